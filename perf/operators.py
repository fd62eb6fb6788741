"""The 8-bit operators of the DoRA path: what each computes, on which sizes it is measured, and its value in 64 bits.

An adapter's frozen weight W0 and the activations that its backward needs are held in 8 bits: e4m3 values with a
power-of-two scale for each block of 128.  A block's scale is 2^e with the smallest e >= -126 for which the block's
largest magnitude times 2^-e is at most 448; the values are the nearest e4m3 values (ties to even) of v * 2^-e.
Activations and gradients have one block per row and 128 columns, the weight one per 128 x 128 tile.  Values that are
not finite are NaN and do not count for the scale.

``run`` calls the framework's operators where ``own`` is true, and their plain form otherwise: elementary torch
operations in fp32, rounded once at the end.  ``exact`` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


# ------------------------------------------------------------------ cases


def listed():
    return [
        # a checkpoint's way there and back: the smallest module, and the input of a ~32B model's MLP down projection
        {"name": "pack_tiny", "op": "pack", "rows": 256, "cols": 512, "dtype": "bf16"},
        {"name": "pack_mlp", "op": "pack", "rows": 10240, "cols": 27648, "dtype": "bf16"},
        # the frozen layer's product: one token as in serving, a short ragged batch of requests, a training batch
        {"name": "linear_token", "op": "linear", "T": 1, "in": 8192, "out": 8192, "dtype": "bf16"},
        {"name": "linear_ragged", "op": "linear", "T": 37, "in": 5120, "out": 27648, "dtype": "fp16"},
        # between the two: the tokens of a few short prompts at once
        {"name": "linear_prompts", "op": "linear", "T": 300, "in": 8192, "out": 8192, "dtype": "bf16"},
        {"name": "linear_wide", "op": "linear", "T": 8192, "in": 8192, "out": 8192, "dtype": "bf16"},
        # its gradient of the input: an attention projection, and the MLP up projection's long contraction
        {"name": "linear_bwd_attn", "op": "linear_bwd", "T": 4096, "in": 4096, "out": 4096, "dtype": "fp16"},
        {"name": "linear_bwd_mlp", "op": "linear_bwd", "T": 10240, "in": 5120, "out": 27648, "dtype": "bf16"},
        # the compose's backward from the 8-bit base: the smallest module, and the 8192-wide one
        {"name": "compose_bwd_tiny", "op": "compose_bwd", "T": 256, "out": 512, "r": 16, "dtype": "fp16", "packed": False},
        {"name": "compose_bwd_wide", "op": "compose_bwd", "T": 8192, "out": 8192, "r": 384, "dtype": "bf16", "packed": True},
        # the gradient of A from the 8-bit input: an odd batch of tokens, and the 8192-wide module
        {"name": "grad_a_attn", "op": "grad_a", "T": 4097, "in": 4096, "r": 64, "dtype": "fp16"},
        {"name": "grad_a_wide", "op": "grad_a", "T": 8192, "in": 8192, "r": 384, "dtype": "bf16"},
    ]


def _size(rng, lo, hi):
    """Spread over the logarithm; a third each of whole blocks of 128, multiples of 8, and any size."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.randrange(3)
    step = (128, 8, 1)[kind]
    return min(hi, max(lo, n // step * step))


def draw(rng):
    op = rng.choice(["pack", "linear", "linear", "linear_bwd", "compose_bwd", "grad_a"])
    dtype = rng.choice(["bf16", "fp16"])
    T, r = _size(rng, 1, 10240), _size(rng, 8, 512)
    out, in_ = _size(rng, 512, 27648), _size(rng, 512, 27648)
    if out * in_ > 27648 * 5120:  # no module is larger than the largest configured one
        in_ = max(512, 27648 * 5120 // out)
    if op == "pack":
        return {"op": op, "rows": T, "cols": in_, "dtype": dtype}
    if op in ("linear", "linear_bwd"):
        return {"op": op, "T": T, "in": in_, "out": out, "dtype": dtype}
    if op == "compose_bwd":
        return {"op": op, "T": T, "out": min(out, 8192), "r": r, "dtype": dtype, "packed": rng.random() < 0.5}
    return {"op": op, "T": T, "in": min(in_, 8192), "r": r, "dtype": dtype}


def work(case):
    """Each input read once and each output written once; 2 operations a multiply-add."""
    op = case["op"]
    if op == "pack":  # the 16-bit rows in, their 8-bit blocks out and in again, the 16-bit rows out
        n = case["rows"] * case["cols"]
        return {"bytes": 6 * n, "flops": 4 * n}
    T, r = case["T"], case.get("r", 0)
    if op in ("linear", "linear_bwd"):
        i, o = case["in"], case["out"]
        return {"bytes": 2 * T * (i + o) + i * o, "flops": 2 * T * i * o}
    if op == "compose_bwd":  # dy in, the base in 8 bits in, d_base out, h and B in, d_B out
        o = case["out"]
        d_base = 4 if case["packed"] else 2  # packed: 8 bits out, in again, and its values out
        return {"bytes": T * o * (2 + 1 + d_base) + 2 * T * r + 4 * o * r + 12 * o, "flops": 2 * T * o * r + 4 * T * o}
    return {"bytes": T * case["in"] + 2 * T * r + 2 * r * case["in"], "flops": 2 * T * case["in"] * r}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV) * scale


def _acts(g, T, n, dt):
    """Activations: unit normal, with one feature in about a hundred twenty times as large, as in trained models."""
    big = torch.rand(n, generator=g, device=DEV) < 0.01
    return (_normal(g, (T, n)) * torch.where(big, 20.0, 1.0)).to(dt)


def _grads(g, T, n, dt):
    """Upstream gradients: normal, each token's of its own size."""
    tok = torch.exp2(_normal(g, (T, 1), 1.5)) * 2.0**-6
    return (_normal(g, (T, n)) * tok).to(dt)


def _scale(r):
    return 32.0 / math.sqrt(r)  # rsLoRA with alpha = 32


def prepare(case, seed):
    g, dt, op = _gen(seed), DT[case["dtype"]], case["op"]
    st = {"case": case, "op": op, "dt": dt}
    if op == "pack":
        st["x"] = _acts(g, case["rows"], case["cols"], dt)
        return st
    T, r = case["T"], case.get("r", 0)
    if op in ("linear", "linear_bwd"):
        W = _normal(g, (case["out"], case["in"]), 0.02).to(dt)
        st["wq"], st["we"] = _pack_weight(W)
        st["x"] = _acts(g, T, case["in"], dt) if op == "linear" else _grads(g, T, case["out"], dt)
        return st
    if op == "compose_bwd":
        o = case["out"]
        st["bq"], st["be"] = _pack(_acts(g, T, o, dt))
        st["dy"] = _grads(g, T, o, dt)
        st["h"], st["B"] = _normal(g, (T, r)).to(dt), _normal(g, (o, r), 0.01).to(dt)
        st["n"] = 1.0 + torch.rand(o, generator=g, device=DEV)
        st["m"] = st["n"] * (1 + _normal(g, (o,), 2.0**-8))
        st["s"] = _scale(r)
        return st
    st["xq"], st["xe"] = _pack(_acts(g, T, case["in"], dt))
    st["dh"] = _grads(g, T, r, dt)
    return st


# ------------------------------------------------------------------ the 8-bit blocks, plain
#
# The layout is the framework's: rows padded with zeros to whole blocks, the exponents as bytes 127 + e in rows of a
# multiple of four; the weight's rows are padded to whole tiles too.


def _up(n, k):
    return -(-n // k) * k


def _bytes(amax):
    """127 + e of blocks with these largest magnitudes (fp32)."""
    frac, ex = torch.frexp(amax)  # amax = frac * 2^ex, frac in [1/2, 1): 448 = 0.875 * 2^9
    e = ex.to(torch.int32) - 9 + (frac > 0.875).to(torch.int32)
    return torch.where(amax > 0, e.clamp(min=-126), torch.full_like(e, -126)) + 127


def _two_to(k):
    """2^k in fp32, exactly, by its exponent field (k from -126 to 127)."""
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _encode(v, e):
    q = v * _two_to(127 - e)
    return torch.where(torch.isfinite(q), q, torch.full_like(q, math.nan)).to(torch.float8_e4m3fn)


def _pack_plain(x):
    T, K = x.shape
    v = torch.zeros((T, _up(K, 128)), device=x.device)
    v[:, :K] = x.float()
    v = v.view(T, -1, 128)
    a = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v)).amax(dim=2)
    e = _bytes(a)
    q = _encode(v, e[:, :, None])
    out = torch.full((T, _up(e.shape[1], 4)), 127, dtype=torch.uint8, device=x.device)
    out[:, : e.shape[1]] = e.to(torch.uint8)
    return q.view(T, -1), out


def _pack_weight_plain(W):
    o, i = W.shape
    op, ip = _up(o, 128), _up(i, 128)
    v = torch.zeros((op, ip), device=W.device)
    v[:o, :i] = W.float()
    v = v.view(op // 128, 128, ip // 128, 128)
    a = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v)).amax(dim=(1, 3))
    e = _bytes(a)
    q = _encode(v, e[:, None, :, None])
    out = torch.full((op // 128, _up(ip // 128, 4)), 127, dtype=torch.uint8, device=W.device)
    out[:, : ip // 128] = e.to(torch.uint8)
    return q.view(op, ip), out


def _unpack(q, e, K):
    T, nb = q.shape[0], q.shape[1] // 128
    s = e[:, :nb].to(torch.int32) - 127
    return (q.float().view(T, nb, 128) * _two_to(s)[:, :, None]).view(T, -1)[:, :K]


def _unpack_weight(q, e, o, i):
    ob, ib = q.shape[0] // 128, q.shape[1] // 128
    s = e[:, :ib].to(torch.int32) - 127
    return (q.float().view(ob, 128, ib, 128) * _two_to(s)[:, None, :, None]).reshape(q.shape)[:o, :i]


def _pack(x):
    if own:
        from dora_fine_tuning_amd import torch_ops

        return torch_ops.q8_pack(x)
    return _pack_plain(x)


def _pack_weight(W):
    if own:
        from dora_fine_tuning_amd import torch_ops

        return torch_ops.q8_pack_weight(W)
    return _pack_weight_plain(W)


def _to(x, dt):
    """One rounding; values past the type's largest are held at it."""
    big = torch.finfo(dt).max
    return x.clamp(-big, big).to(dt)


# ------------------------------------------------------------------ one pass


def _compose_bwd(dy, base, h, B, m, n, s, add_base):
    """d_base, E = dy^T h (so d_B = g s E) and d_mag, the token sums of d_mag in 64 bits."""
    g = m / n
    d = dy.float()
    d_base = (g if add_base else (m - n) / n) * d
    E = d.t() @ h
    t = (d * base).sum(dim=0, dtype=torch.float64) + s * (B.double() * (d.t().double() @ h.double())).sum(dim=1)
    return d_base, (g * s)[:, None] * E, (t / n.double()).float()


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    from dora_fine_tuning_amd import torch_ops as F

    c, op, dt = st["case"], st["op"], st["dt"]
    if op == "pack":
        q, e = F.q8_pack(st["x"])
        return F.q8_unpack(q, e, c["cols"], dt)
    if op == "linear":
        q, e = F.q8_pack(st["x"])
        return F.q8_linear(q, e, st["wq"], st["we"], c["out"], dt)
    if op == "linear_bwd":
        q, e = F.q8_pack(st["x"])
        return F.q8_linear_backward(q, e, st["wq"], st["we"], c["in"], dt)
    if op == "compose_bwd":
        args = (st["dy"], st["bq"], st["be"], st["h"], st["B"], st["m"], st["n"], st["s"], True)
        if c["packed"]:
            q, e, d_B, d_mag = F.q8_lora_compose_backward_packed(*args)
            return {"d_base": F.q8_unpack(q, e, c["out"], dt), "d_B": d_B, "d_mag": d_mag}
        d_base, d_B, d_mag = F.q8_lora_compose_backward(*args, True)
        return {"d_base": d_base, "d_B": d_B, "d_mag": d_mag}
    return F.q8_grad_a(st["dh"], st["xq"], st["xe"], c["in"])


def _run_plain(st):
    c, op, dt = st["case"], st["op"], st["dt"]
    if op == "pack":
        return _to(_unpack(*_pack_plain(st["x"]), c["cols"]), dt)
    if op == "linear":
        x = _unpack(*_pack_plain(st["x"]), c["in"])
        return (x @ _unpack_weight(st["wq"], st["we"], c["out"], c["in"]).t()).to(dt)
    if op == "linear_bwd":
        g = _unpack(*_pack_plain(st["x"]), c["out"])
        return (g @ _unpack_weight(st["wq"], st["we"], c["out"], c["in"])).to(dt)
    if op == "compose_bwd":
        base = _unpack(st["bq"], st["be"], c["out"])
        d_base, d_B, d_mag = _compose_bwd(st["dy"], base, st["h"].float(), st["B"], st["m"], st["n"], st["s"], True)
        if c["packed"]:
            d_base = _to(_unpack(*_pack_plain(d_base), c["out"]), dt)
        return {"d_base": d_base.to(dt), "d_B": d_B.to(dt), "d_mag": d_mag}
    return (st["dh"].float().t() @ _unpack(st["xq"], st["xe"], c["in"])).to(dt)


# ------------------------------------------------------------------ in 64 bits


def _pow2(k):
    """2^k in fp64, exactly (whole k, in fp64 or an integer type)."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _nearest(v, dims, shape):
    """The values that v's blocks (`dims` of v viewed as `shape`) are held as, from the definition."""
    b = v.view(shape)
    a = torch.where(torch.isfinite(b), b.abs(), torch.zeros_like(b)).amax(dim=dims, keepdim=True)
    e = torch.ceil(torch.log2(a.clamp(min=1e-300) / 448.0)).clamp(min=-126.0)
    # the logarithm may be off by one next to a power of two: the smallest e with a <= 448 * 2^e
    e = torch.where(a * _pow2(1 - e) <= 448.0, (e - 1).clamp(min=-126.0), e)
    e = torch.where(a * _pow2(-e) > 448.0, e + 1, e)
    s = _pow2(e)
    w = b / s
    # e4m3 has 3 bits after the leading one and nothing finer than 2^-9
    _, k = torch.frexp(w)
    step = _pow2((k - 4).clamp(min=-9))
    w = torch.where(torch.isfinite(w), torch.round(w / step) * step, torch.full_like(w, math.nan))
    return (w * s).view(v.shape)


def _held(x):
    """Rows of x in 8 bits, as fp64 values."""
    T, K = x.shape
    v = torch.zeros((T, _up(K, 128)), dtype=torch.float64, device=x.device)
    v[:, :K] = x
    return _nearest(v, (2,), (T, v.shape[1] // 128, 128))[:, :K]


def _held_weight(q, e, o, i):
    s = _pow2(e[:, : q.shape[1] // 128].long() - 127)
    return (q.to(torch.float32).double() * s.repeat_interleave(128, dim=0).repeat_interleave(128, dim=1))[:o, :i]


def _held_rows(q, e, K):
    e = e[:, : q.shape[1] // 128].long() - 127
    return (q.to(torch.float32).double() * _pow2(e).repeat_interleave(128, dim=1))[:, :K]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    c, op = st["case"], st["op"]
    big = torch.finfo(st["dt"]).max
    if op == "pack":
        return _held(st["x"]).clamp(-big, big)
    if op in ("linear", "linear_bwd"):
        W = _held_weight(st["wq"], st["we"], c["out"], c["in"])
        return _held(st["x"]) @ (W.t() if op == "linear" else W)
    if op == "grad_a":
        return st["dh"].double().t() @ _held_rows(st["xq"], st["xe"], c["in"])
    s, m, B, dy = st["s"], st["m"].double(), st["B"].double(), st["dy"].double()
    n, h, base = st["n"].double(), st["h"].double(), _held_rows(st["bq"], st["be"], c["out"])
    g = m / n
    d_base = _held(g * dy).clamp(-big, big) if c["packed"] else g * dy
    d_B = (g * s)[:, None] * (dy.t() @ h)
    return {"d_base": d_base, "d_B": d_B, "d_mag": (dy * (base + s * (h @ B.t()))).sum(dim=0) / n}
