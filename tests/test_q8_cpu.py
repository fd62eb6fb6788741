"""The 8-bit operators without a GPU: pins of their oracle, the eager tier
against it, the layer's gradients, and the entry points' refusals."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from dora_fine_tuning_amd import binding
from oracle import dora_oracle as O
from oracle import q8_oracle as Q

F = pytest.importorskip("dora_fine_tuning_amd.torch_ops")
LIB = binding.LIB
OK, INVALID, UNSUPPORTED = binding.DORA_OK, binding.DORA_INVALID_ARG, binding.DORA_UNSUPPORTED


def _u8(q):
    return q.view(torch.uint8).numpy()


# ------------------------------------------------------------------ the oracle's pins


def test_oracle_table_is_the_format():
    """All 256 bytes against torch's own decoding of the type."""
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(Q.E4M3))
    ok = ~np.isnan(t)
    assert np.array_equal(t[ok], Q.E4M3[ok]) and Q.E4M3[126] == 448.0


def test_oracle_rounding_by_exact_distance():
    """Nearest and ties to even, by exact rational distances to every value of the type."""
    rng = np.random.default_rng(3)
    mids = (Q._POS[:-1] + Q._POS[1:]) / 2  # every tie
    v = np.concatenate([mids, -mids, Q._POS, mids * (1 + 2.0**-40), mids * (1 - 2.0**-40),
                        rng.uniform(-448, 448, 200), rng.normal(0, 2.0**-7, 200)])
    v = v[np.abs(v) <= 448]
    got = Q.nearest_byte(v)
    vals = [(b, Fraction(float(Q._POS[b]))) for b in range(127)]
    for x, b in zip(v, got):
        a = abs(Fraction(float(x)))
        best = min(vals, key=lambda p: (abs(p[1] - a), p[0] & 1))
        assert (int(b) & 127) == best[0], (x, b, best)
        assert (int(b) >> 7) == int(np.signbit(x))


def test_oracle_exponent_is_the_smallest():
    rng = np.random.default_rng(4)
    a = np.concatenate([[0.0, 448.0, 449.0, 896.0, 2.0**-140, 3.3895313892515355e38],
                        np.exp2(rng.uniform(-130, 127, 200))])
    got = Q._exponents(a)
    for x, e in zip(a, got):
        assert e == Q.block_exponent(x)
        assert x <= 448 * 2.0**e and (e == -126 or x > 448 * 2.0 ** (e - 1))


def test_oracle_products_by_differences():
    """linear is bilinear, so its gradients are exact differences: dx, and d_A
    as the gradient of sum(dh * (x A^T))."""
    rng = np.random.default_rng(5)
    x, W = rng.normal(size=(4, 6)), rng.normal(size=(5, 6))
    dy, dx = rng.normal(size=(4, 5)), rng.normal(size=(4, 6))
    diff = (np.sum(dy * Q.linear(x + dx, W)) - np.sum(dy * Q.linear(x - dx, W))) / 2
    assert np.isclose(diff, np.sum(Q.linear_bwd(dy, W) * dx), rtol=1e-12)
    A, dA, dh = rng.normal(size=(3, 6)), rng.normal(size=(3, 6)), rng.normal(size=(4, 3))
    diff = (np.sum(dh * (x @ (A + dA).T)) - np.sum(dh * (x @ (A - dA).T))) / 2
    assert np.isclose(diff, np.sum(Q.grad_a(dh, x) * dA), rtol=1e-12)


# ------------------------------------------------------------------ the eager tier


def special_rows(dtype):
    """Rows with what a block can hold: zeros, not-finite values, the largest and
    smallest of the type, values at the limit between two exponents."""
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    x = torch.zeros(8, 300, dtype=torch.float64)
    g = torch.Generator().manual_seed(2)
    x[1] = torch.randn(300, generator=g, dtype=torch.float64)
    x[1, 5], x[1, 200] = float("inf"), float("nan")
    x[2, :128] = float("-inf")
    x[3] = torch.randn(300, generator=g, dtype=torch.float64) * tiny
    x[4] = torch.linspace(-1, 1, 300, dtype=torch.float64) * big
    x[5, 0], x[5, 1], x[5, 128], x[5, 256] = 448.0, -0.0, 450.0, 224.0
    x[6] = torch.exp2(torch.linspace(-20, 8, 300, dtype=torch.float64))
    x[7] = tiny / 4
    return x.clamp(-big, big).where(torch.isfinite(x), x).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 1), (3, 128), (5, 130), (7, 513)])
def test_eager_pack_is_the_oracle(dtype, shape):
    g = torch.Generator().manual_seed(shape[1])
    x = (torch.randn(shape, generator=g) * torch.exp2(torch.randn(shape[0], 1, generator=g) * 6)).to(dtype)
    for xs in ([x] if dtype == torch.float32 else [x, special_rows(dtype)]):
        q, e = F.q8_pack(xs)
        rq, re_ = Q.pack_rows(O.as_f64(xs))
        nan = Q.E4M3[_u8(q)]
        assert np.array_equal(np.isnan(nan), np.isnan(Q.E4M3[rq]))
        assert np.array_equal(np.where(np.isnan(nan), 0, _u8(q)), np.where(np.isnan(nan), 0, rq))
        assert np.array_equal(e.numpy(), re_)
        wq, we = F.q8_pack_weight(xs)
        rwq, rwe = Q.pack_weight(O.as_f64(xs))
        ok = ~np.isnan(Q.E4M3[rwq])
        assert np.array_equal(_u8(wq)[ok], rwq[ok]) and np.array_equal(we.numpy(), rwe)


def test_eager_products_are_the_oracle():
    g = torch.Generator().manual_seed(8)
    x, W = torch.randn(9, 200, generator=g).bfloat16(), (torch.randn(150, 200, generator=g) * 0.02).bfloat16()
    dy = torch.randn(9, 150, generator=g).bfloat16()
    wq, we = F.q8_pack_weight(W)
    Wh = Q.held_weight(*Q.pack_weight(O.as_f64(W)), 150, 200)
    xh, dh = Q.held_rows(*Q.pack_rows(O.as_f64(x)), 200), Q.held_rows(*Q.pack_rows(O.as_f64(dy)), 150)
    # one rounding to bf16, and fp32 sums of at most 200 products
    y = F.q8_linear(*F.q8_pack(x), wq, we, 150, torch.bfloat16).double().numpy()
    assert np.all(np.abs(y - Q.linear(xh, Wh)) <= 2.0**-8 * np.abs(y) + 200 * 2.0**-24 * (np.abs(xh) @ np.abs(Wh).T))
    dx = F.q8_linear_backward(*F.q8_pack(dy), wq, we, 200, torch.bfloat16).double().numpy()
    assert np.all(np.abs(dx - Q.linear_bwd(dh, Wh)) <= 2.0**-8 * np.abs(dx) + 150 * 2.0**-24 * (np.abs(dh) @ np.abs(Wh)))


def ste_reference(x, W, A, B, m, s, dy, q8_weight, detach):
    """The layer's outputs and gradients in fp64 from their formulas: base from
    the held x with an 8-bit weight, the backward from the held x, base and (with
    an 8-bit weight) d_base; n by autograd where it is not detached."""
    x, W, A, B, m, dy = (O.as_f64(t) for t in (x, W, A, B, m, dy))
    held = lambda v: Q.held_rows(*Q.pack_rows(v), v.shape[1])
    V = W + s * (B @ A)
    n = np.linalg.norm(V, axis=1)
    g = m / n
    xh, h = held(x), x @ A.T
    base = (xh if q8_weight else x) @ W.T
    bh, d_base = held(base), g * dy
    d_h = (g * s * dy) @ B
    out = dict(y=g * base + g * s * (h @ B.T), d_mag=(dy * (bh + s * h @ B.T)).sum(0) / n, d_B=(g * s * dy).T @ h,
               d_A=d_h.T @ xh, dx=(held(d_base) if q8_weight else d_base) @ W + d_h @ A)
    if not detach:
        dV = (-(g * out["d_mag"]) / n)[:, None] * V
        out["d_A"] = out["d_A"] + s * B.T @ dV
        out["d_B"] = out["d_B"] + s * dV @ A.T
    return out


def layer_case(dtype, device, T, i, o, r, seed=0, **kw):
    torch.manual_seed(seed)
    layer = F.DoRALinear(i, o, r, dtype=dtype, device=device, **kw)
    with torch.no_grad():
        layer.lora_B.normal_(0.0, 0.02)
        layer.magnitude.mul_(1.0 + 0.01 * torch.randn_like(layer.magnitude))
    x = torch.randn(T, i, device=device).to(dtype)
    return layer, x, torch.randn(T, o, device=device).to(dtype)


def check_layer(layer, x, dy, tol, tol_mag):
    W = layer.weight
    if layer.q8_weight:
        W = F.q8_unpack_weight(*layer._packed_weight(), layer.out_features, layer.in_features, x.dtype)
    ref = ste_reference(x, W, layer.lora_A, layer.lora_B, layer.magnitude, layer.s, dy, layer.q8_weight,
                        layer.detach_norm)
    x = x.clone().requires_grad_()
    y = layer(x)
    dx, dA, dB, dm = torch.autograd.grad(y, (x, layer.lora_A, layer.lora_B, layer.magnitude), dy)
    got = dict(y=y, dx=dx, d_A=dA, d_B=dB, d_mag=dm)
    for k, v in got.items():
        v = v.detach().double().cpu().numpy()
        rel = np.linalg.norm(v - ref[k]) / np.linalg.norm(ref[k])
        assert rel <= (tol_mag if k == "d_mag" else tol), (k, rel)


@pytest.mark.parametrize("kw", [dict(q8_weight=True), dict(q8_checkpoint=True),
                                dict(q8_weight=True, detach_norm=False)])
def test_eager_layer_gradients(kw):
    layer, x, dy = layer_case(torch.float32, None, 21, 200, 150, 8, **kw)
    # fp32 throughout; a value of base or d_base next to a step of the 8-bit type
    # may land on the other side of it, one step (2^-3 of the value) in few of the
    # 21 or 150 terms of a sum
    check_layer(layer, x, dy, 1e-3, 2e-2)
    with torch.no_grad():
        y0 = layer(x)
    assert torch.equal(y0, layer(x).detach())


def packed_operator_calls(device, dtype):
    """Every 8-bit operator with the positions of its arguments that a gradient could reach."""
    x, W = torch.randn(5, 200, device=device).to(dtype), torch.randn(140, 200, device=device).to(dtype)
    dy, h, B = (torch.randn(*s, device=device).to(dtype) for s in ((5, 140), (5, 8), (140, 8)))
    m, n = torch.rand(140, device=device) + 1, torch.rand(140, device=device) + 1
    (xq, xe), (wq, we), (bq, be) = F.q8_pack(x), F.q8_pack_weight(W), F.q8_pack(dy)
    return [(F.q8_pack, (x,), (0,)), (F.q8_pack_weight, (W,), (0,)), (F.q8_unpack, (xq, xe, 200, dtype), (0,)),
            (F.q8_unpack_weight, (wq, we, 140, 200, dtype), (0,)),
            (F.q8_linear, (xq, xe, wq, we, 140, dtype), (0, 2)),
            (F.q8_linear_backward, (bq, be, wq, we, 200, dtype), (0, 2)),
            (F.q8_lora_compose_backward, (dy, bq, be, h, B, m, n, 1.0, True, True), (0, 1, 3, 4, 5, 6)),
            (F.q8_lora_compose_backward_packed, (dy, bq, be, h, B, m, n, 1.0, True), (0, 1, 3, 4, 5, 6)),
            (F.q8_grad_a, (h, xq, xe, 200), (0, 1))]


def check_gradients_are_refused(device, dtype):
    for op, args, where in packed_operator_calls(device, dtype):
        op(*args)
        for i in where:
            with_grad = [a.detach().requires_grad_() if j == i else a for j, a in enumerate(args)]
            with pytest.raises(RuntimeError, match="no gradient of its own"):
                op(*with_grad)
            with torch.no_grad():
                out = op(*with_grad)
            assert not any(t.requires_grad for t in (out if isinstance(out, tuple) else (out,)))


def test_packed_operators_refuse_gradients():
    check_gradients_are_refused("cpu", torch.float32)


def check_layer_outputs(device, dtype):
    """Of q8_layer's outputs y alone has a gradient, and a second backward is refused."""
    layer, x, dy = layer_case(dtype, device, 6, 200, 150, 8, q8_weight=True)
    x.requires_grad_()
    wq, we = layer._packed_weight()
    y, *kept = F.q8_layer(x, layer.lora_A, layer.lora_B, layer.magnitude, layer.weight_norm(), wq, we, layer.s)
    assert y.requires_grad and not any(t.requires_grad for t in kept)
    with pytest.raises(RuntimeError, match="no gradient of its own"):
        torch.autograd.grad(y, x, dy.requires_grad_(), create_graph=True)


def test_layer_outputs():
    check_layer_outputs(None, torch.float32)


def test_layer_takes_another_layers_parameter():
    lin = torch.nn.Linear(200, 150, bias=False)
    layer = F.DoRALinear(200, 150, 8, dtype=torch.float32, weight=lin.weight, q8_weight=True)
    assert not layer.weight_q.requires_grad and not layer.magnitude.grad_fn
    assert F.DoRALinear(200, 150, 8, q8_weight=True)(torch.randn(0, 200).bfloat16()).shape == (0, 150)


def test_layer_holds_the_weight_in_bytes():
    layer = F.DoRALinear(200, 150, 8, dtype=torch.bfloat16, q8_weight=True)
    assert layer.weight is None and layer.weight_q.dtype == torch.uint8 and layer.weight_q.shape == (256, 256)
    other = F.DoRALinear(200, 150, 8, dtype=torch.bfloat16, q8_weight=True)
    state = layer.state_dict()
    state.pop("weight_sqnorm", None)
    other.load_state_dict(state, strict=False)
    assert torch.equal(other.weight_q, layer.weight_q) and torch.equal(other.weight_e, layer.weight_e)


def test_layer_compiles_without_graph_breaks():
    for kw in (dict(q8_weight=True), dict(q8_checkpoint=True)):
        layer, x, dy = layer_case(torch.bfloat16, None, 5, 200, 150, 8, **kw)
        layer.refresh_weight_cache()
        f = torch.compile(layer, fullgraph=True, backend="aot_eager")
        xa, xb = x.clone().requires_grad_(), x.clone().requires_grad_()
        ga, gb = torch.autograd.grad(layer(xa), xa, dy)[0], torch.autograd.grad(f(xb), xb, dy)[0]
        assert torch.equal(ga, gb)


# ------------------------------------------------------------------ refusals, before any launch

P = 1 << 20  # fake, never dereferenced
FAR = [(k + 1) << 44 for k in range(16)]


def _status(ret, want, fragment):
    assert ret == want, (ret, binding.dora_last_error())
    assert fragment in binding.dora_last_error(), binding.dora_last_error()


def test_pack_refusals():
    for fn in (LIB.dora_q8_pack, LIB.dora_q8_pack_weight):
        _status(fn(P, 8, 8, 5, P * 2, P * 3, None), UNSUPPORTED, "dtype")
        _status(fn(P, -1, 8, 0, P * 2, P * 3, None), INVALID, "negative")
        _status(fn(None, 8, 8, 0, P * 2, P * 3, None), INVALID, "NULL")
        _status(fn(P, 8, 8, 0, None, P * 3, None), INVALID, "NULL")
        _status(fn(P, 8, 8, 0, P * 2 + 8, P * 3, None), INVALID, "alignment")
        _status(fn(P, 8, 8, 0, P * 2, P * 3 + 2, None), INVALID, "alignment")
        _status(fn(P, 8, 8, 0, P, P * 3, None), INVALID, "overlaps")
        _status(fn(P, 8, 8, 0, P * 2, P * 2 + 64, None), INVALID, "overlaps")
        _status(fn(FAR[0], 8, 1 << 23, 0, FAR[1], FAR[2], None), UNSUPPORTED, "beyond")
        _status(fn(FAR[0], (1 << 22) - 128, (1 << 22) - 128, 0, FAR[1], FAR[2], None), UNSUPPORTED, "blocks")
        assert fn(None, 0, 8, 0, None, None, None) == OK and fn(None, 8, 0, 0, None, None, None) == OK
    _status(LIB.dora_q8_pack(FAR[0], 1 << 31, 8, 0, FAR[1], FAR[2], None), UNSUPPORTED, "beyond")
    u = LIB.dora_q8_unpack
    _status(u(P, P * 2, 8, 8, 0, 9, P * 3, None), UNSUPPORTED, "dtype")
    _status(u(P, P * 2, 8, -8, 1, 0, P * 3, None), INVALID, "negative")
    _status(u(P, None, 8, 8, 1, 0, P * 3, None), INVALID, "NULL")
    _status(u(P, P * 2, 8, 8, 0, 0, None, None), INVALID, "NULL")
    _status(u(P, P * 2, 8, 8, 0, 0, P + 16, None), INVALID, "overlaps")
    assert u(None, None, 0, 8, 0, 0, None, None) == OK


@pytest.mark.parametrize("name", ["fwd", "bwd"])
def test_linear_refusals(name):
    fn = getattr(LIB, f"dora_q8_linear_{name}")
    query = LIB.dora_q8_linear_workspace_bytes if name == "fwd" else LIB.dora_q8_linear_bwd_workspace_bytes

    def call(xq=FAR[0], xe=FAR[1], wq=FAR[2], we=FAR[3], T=200, out=256, in_=4096, dt=0, y=FAR[4], ws=FAR[5],
             wsb=1 << 40):
        return fn(xq, xe, wq, we, T, out, in_, dt, y, ws, wsb, None)

    _status(call(dt=2), UNSUPPORTED, "dtype")
    _status(call(T=-1), INVALID, "negative")
    _status(call(out=1 << 22), UNSUPPORTED, "beyond")
    _status(call(y=None), INVALID, "NULL")
    _status(call(y=FAR[4] + 1), INVALID, "alignment")
    _status(call(xq=None), INVALID, "packed rows")
    _status(call(xe=FAR[1] + 1), INVALID, "alignment")
    _status(call(wq=FAR[2] + 8), INVALID, "packed weight")
    _status(call(y=FAR[2]), INVALID, "overlaps")
    _status(call(y=FAR[0] + 2), INVALID, "overlaps")
    # a split contraction needs its workspace
    T, out, in_ = (200, 256, 4096) if name == "fwd" else (200, 4096, 256)
    need = query(T, out, in_)
    assert need > 0
    _status(call(T=T, out=out, in_=in_, wsb=need - 1), INVALID, "workspace of")
    _status(call(T=T, out=out, in_=in_, ws=None), INVALID, "workspace is NULL")
    _status(call(T=T, out=out, in_=in_, ws=FAR[4]), INVALID, "overlaps")
    _status(call(T=(1 << 31) - 1, out=(1 << 22) - 128, in_=(1 << 22) - 128, xe=1 << 60, wq=1 << 59, we=1 << 58, y=1 << 61), UNSUPPORTED, "workgroups")
    assert call(T=0, xq=None, y=None) == OK
    assert query(0, 8, 8) == 0 and query(-1, 8, 8) == 0 and query(8, 1 << 24, 8) == 0


def test_compose_bwd_refusals():
    need = LIB.dora_q8_lora_compose_bwd_workspace_bytes(64, 16, 8)
    assert need > 0

    def call(dt=0, T=64, out=16, r=8, wsb=1 << 40, **kw):
        a = dict(zip("dy bq be h B mag norm d_base dq de d_B d_mag ws".split(), FAR), **kw)
        return LIB.dora_q8_lora_compose_bwd(a["dy"], a["bq"], a["be"], a["h"], a["B"], a["mag"], a["norm"], 1.0, T, out,
                                            r, dt, 0, a["d_base"], a["dq"], a["de"], a["d_B"], a["d_mag"], a["ws"],
                                            wsb, None)

    _status(call(dt=7), UNSUPPORTED, "dtype")
    _status(call(r=-1), INVALID, "negative")
    _status(call(r=(1 << 20) + 8), UNSUPPORTED, "2^20")
    _status(call(d_mag=None), INVALID, "d_mag")
    _status(call(dy=None), INVALID, "dy")
    _status(call(dy=FAR[0] + 2), INVALID, "aligned")
    _status(call(bq=None), INVALID, "packed base")
    _status(call(be=FAR[2] + 2), INVALID, "alignment")
    _status(call(h=None), INVALID, "h is NULL")
    _status(call(d_B=None), INVALID, "d_B")
    _status(call(h=FAR[3] + 8), INVALID, "alignment")
    _status(call(dq=None), INVALID, "together")
    _status(call(wsb=need - 1), INVALID, "workspace of")
    _status(call(ws=None), INVALID, "workspace is NULL")
    _status(call(dq=FAR[1]), INVALID, "overlaps")
    _status(call(d_base=FAR[0]), INVALID, "overlaps")
    _status(call(d_mag=FAR[5]), INVALID, "overlaps")
    _status(call(T=(1 << 31) - 1, out=(1 << 22) - 128, wsb=1 << 62), UNSUPPORTED, "workgroups")
    assert LIB.dora_q8_lora_compose_bwd(*[None] * 7, 1.0, 8, 0, 8, 0, 0, *[None] * 6, 0, None) == OK
    assert LIB.dora_q8_lora_compose_bwd_workspace_bytes(8, 0, 8) == 0


def test_grad_a_refusals():
    need = LIB.dora_q8_grad_a_workspace_bytes(64, 128, 8)

    def call(dh=FAR[0], xq=FAR[1], xe=FAR[2], T=64, in_=128, r=8, dt=0, dA=FAR[3], ws=FAR[4], wsb=1 << 40):
        return LIB.dora_q8_grad_a(dh, xq, xe, T, in_, r, dt, dA, ws, wsb, None)

    _status(call(dt=3), UNSUPPORTED, "dtype")
    _status(call(T=-2), INVALID, "negative")
    _status(call(r=1 << 21), UNSUPPORTED, "2^20")
    _status(call(dA=None), INVALID, "d_A")
    _status(call(dh=FAR[0] + 4), INVALID, "aligned")
    _status(call(xq=None), INVALID, "packed x")
    _status(call(wsb=need - 1), INVALID, "workspace of")
    _status(call(ws=FAR[4] + 4), INVALID, "aligned")
    _status(call(dA=FAR[0] + 2), INVALID, "overlaps")
    _status(call(T=(1 << 31) - 1, in_=(1 << 22) - 128, wsb=1 << 62), UNSUPPORTED, "workgroups")
    assert call(r=0, dh=None, dA=None) == OK and call(in_=0, xq=None) == OK


def test_binding_refuses_wrong_layouts():
    q, e = F.q8_pack(torch.zeros(4, 200).bfloat16())
    with pytest.raises(ValueError, match="HIP device"):
        binding.dora_q8_pack(torch.zeros(4, 200).bfloat16())
    with pytest.raises(ValueError, match="HIP device"):
        binding.dora_q8_unpack(q, e, 4, 200, torch.bfloat16)
    with pytest.raises(ValueError, match="dtype"):
        binding.dora_q8_unpack(q, e, 4, 200, torch.float32)


def test_workspace_queries_do_not_shrink_with_padding():
    # odd sizes add the padded copies; multiples of 8 add none
    a = LIB.dora_q8_lora_compose_bwd_workspace_bytes(1000, 1000, 16)
    b = LIB.dora_q8_lora_compose_bwd_workspace_bytes(1000, 999, 15)
    assert b >= a + 1000 * 1000 * 2 + 1000 * 16 * 2 - 16 * 4 * 1000
    assert LIB.dora_q8_linear_workspace_bytes(8192, 8192, 8192) == 0
    assert LIB.dora_q8_linear_workspace_bytes(1, 8192, 8192) == 0
