"""The 4-bit weight without a GPU: pins of its oracle, the eager tier against it,
the layer's gradients, and the entry points' refusals."""
import concurrent.futures
from fractions import Fraction

import numpy as np
import pytest
import torch

from dora_fine_tuning_amd import binding
from oracle import dora_oracle as O
from oracle import q4_oracle as Q

F = pytest.importorskip("dora_fine_tuning_amd.torch_ops")
LIB = binding.LIB
OK, INVALID, UNSUPPORTED = binding.DORA_OK, binding.DORA_INVALID_ARG, binding.DORA_UNSUPPORTED
P = 1 << 40  # addresses that no refused call touches
FAR = [P * (i + 1) for i in range(8)]


def special_weight(dtype):
    """Every border of the rounding at several scales, the ends of the exponents'
    range, zeros of both signs, values that are not finite."""
    borders = [0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 6.5, 7.0]
    rows = []
    for e in (-24, -23, -22, -9, 0, 5, 12, 13):
        v = np.array(borders + [-b for b in borders[1:16]])
        rows.append(v * 2.0**e)  # 32 values: one block
        rows.append(v[::-1] * 2.0**e * (1 + 2.0**-7))
        rows.append(np.where(v == 7.0, 7.0 * (1 + 2.0**-7), v) * 2.0**e)  # just past the limit
    rows.append(np.full(32, 2.0**-40))
    rows.append(np.full(32, -0.0))
    rows.append(np.where(np.arange(32) == 3, 60000.0, 1.0))
    w = torch.tensor(np.array(rows), dtype=torch.float64).to(dtype)
    w = torch.cat((w, w[:3], w[:1] * 0), dim=0).repeat(1, 3)  # three blocks a row, the last column tile half full
    w[-2, 40], w[-3, 0], w[-4, 95] = float("nan"), float("inf"), float("-inf")
    return w


def rnd(seed, shape, dtype, scale=1.0, spread=0.0):
    rng = np.random.default_rng(seed)
    v = rng.standard_normal(shape) * scale
    if spread:
        v = v * np.exp2(rng.standard_normal((shape[0], 1)) * spread)
    return torch.from_numpy(v.astype(np.float32)).to(dtype)


# ------------------------------------------------------------------ the oracle's pins


def test_oracle_table_is_the_format():
    assert Q.E2M1[:8].tolist() == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    assert Q.E2M1[8:].tolist() == [-v for v in Q.E2M1[:8]]


def test_oracle_rounding_by_exact_distance():
    rng = np.random.default_rng(3)
    mids = (Q.E2M1[:7] + Q.E2M1[1:8]) / 2
    v = np.concatenate([mids, -mids, Q.E2M1, mids * (1 + 2.0**-40), mids * (1 - 2.0**-40), rng.uniform(-7, 7, 300)])
    got = Q.nearest_code(v)
    for x, c in zip(v, got):
        a = min(abs(Fraction(float(x))), Fraction(6))
        want = min(range(8), key=lambda k: (abs(Fraction(float(Q.E2M1[k])) - a), k & 1))
        assert (int(c) & 7) == want and (int(c) >> 3) == int(np.signbit(x)), (x, c)


def test_oracle_exponent_is_the_smallest():
    for a in [0.0, 7.0, 7.0001, 14.0, 2.0**-30, 7 * 2.0**-23, 7.01 * 2.0**-23, 7 * 2.0**13, 1e30, 0.02, 3.5, 3.51]:
        e = Q.block_exponent(a)
        assert -23 <= e <= 13 and (a <= 7 * 2.0**e or e == 13) and (e == -23 or a > 7 * 2.0 ** (e - 1))


def test_every_held_value_is_exact_in_both_types():
    v = np.outer(2.0 ** np.arange(-23, 14), Q.E2M1).ravel()
    for dt in (torch.bfloat16, torch.float16):
        assert np.array_equal(torch.from_numpy(v).to(dt).double().numpy(), v)


# ------------------------------------------------------------------ the eager tier


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 1), (1, 64), (3, 63), (33, 65), (70, 200), (64, 128)])
def test_eager_pack_is_the_oracle(shape, dtype):
    W = rnd(shape[0] * 7 + shape[1], shape, dtype, spread=6.0)
    q, e = F.q4_pack_weight(W)
    rq, re_ = Q.pack(O.as_f64(W))
    assert np.array_equal(q.numpy(), rq) and np.array_equal(e.numpy(), re_)
    for dt in (dtype, torch.float32, torch.float64):
        got = F.q4_unpack_weight(q, e, *shape, dt).double().numpy()
        assert np.array_equal(got, Q.held(O.as_f64(W)), equal_nan=True)  # (fp16 has infinities here)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_eager_pack_special_values(dtype):
    W = special_weight(dtype)
    q, e = F.q4_pack_weight(W)
    rq, re_ = Q.pack(O.as_f64(W))
    assert np.array_equal(q.numpy(), rq) and np.array_equal(e.numpy(), re_)
    held = Q.held(O.as_f64(W))
    assert np.isnan(held).any() and np.array_equal(
        F.q4_unpack_weight(q, e, *W.shape, dtype).double().numpy(), held, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,out,in_", [(1, 1, 1), (5, 70, 200), (9, 32, 64), (0, 40, 8), (4, 0, 8), (4, 8, 0)])
def test_eager_products(T, out, in_, dtype):
    W = rnd(1, (out, in_), dtype, 0.02)
    q, e = F.q4_pack_weight(W)
    held = Q.held(O.as_f64(W)) if W.numel() else np.zeros((out, in_))
    half = torch.finfo(dtype).eps / 2
    for x, M, op in ((rnd(2, (T, in_), dtype), held.T, lambda v: F.q4_linear(v, q, e, out)),
                     (rnd(3, (T, out), dtype), held, lambda v: F.q4_linear_backward(v, q, e, in_))):
        want, mass, y = O.as_f64(x) @ M, np.abs(O.as_f64(x)) @ np.abs(M), op(x)
        assert y.dtype == dtype and tuple(y.shape) == want.shape
        tol = half * np.abs(want) + M.shape[0] * 2.0**-23 * mass + 2.0**-25
        assert np.all(np.abs(y.double().numpy() - want) <= tol)


def test_gradients_are_the_formulas_and_the_differences():
    """y is linear in x: its gradient is dy W, equal to the differences of the loss; and so is the gradient's own."""
    W = rnd(5, (24, 40), torch.float32, 0.1)
    q, e = F.q4_pack_weight(W)
    held = torch.from_numpy(Q.held(O.as_f64(W)))
    x = rnd(6, (3, 40), torch.float32).requires_grad_()
    dy = rnd(7, (3, 24), torch.float32)
    y = F.q4_linear(x, q, e, 24)
    (dx,) = torch.autograd.grad(y, x, dy)
    torch.testing.assert_close(dx, (dy.double() @ held).float(), rtol=1e-5, atol=1e-6)
    for i, j in ((0, 0), (2, 39), (1, 17)):
        d = torch.zeros_like(x)
        d[i, j] = 1.0
        step = ((F.q4_linear(x.detach() + d, q, e, 24) - F.q4_linear(x.detach() - d, q, e, 24)) * dy).sum() / 2
        assert abs(float(step - dx[i, j])) <= 1e-4
    # create_graph: d/dx sum((W^T W x)^2)
    (g,) = torch.autograd.grad(0.5 * F.q4_linear(x, q, e, 24).square().sum(), x, create_graph=True)
    (h,) = torch.autograd.grad(0.5 * g.square().sum(), x)
    G = held.T @ held
    torch.testing.assert_close(h.double(), x.detach().double() @ G @ G, rtol=1e-4, atol=1e-5)


def test_no_gradient_of_the_weight_and_none_where_none_is_asked():
    q, e = F.q4_pack_weight(rnd(1, (32, 64), torch.float32))
    x = torch.zeros(2, 64)
    assert not F.q4_linear(x, q, e, 32).requires_grad
    with torch.no_grad():
        assert not F.q4_linear(x.requires_grad_(), q, e, 32).requires_grad
    for op, args in ((F.q4_pack_weight, (torch.zeros(4, 4, requires_grad=True),)),):
        with pytest.raises(RuntimeError, match="no gradient"):
            op(*args)
    import torch.autograd.forward_ad as fwad

    with fwad.dual_level():
        for g in (False, True):
            dual = fwad.make_dual(torch.zeros(2, 64, requires_grad=g), torch.ones(2, 64))
            with pytest.raises(RuntimeError, match="q4_linear has no"):
                F.q4_linear(dual, q, e, 32)


def check_compiled(device, dtype):
    q, e = F.q4_pack_weight(rnd(1, (40, 72), dtype).to(device))
    x = rnd(2, (6, 72), dtype).to(device).requires_grad_()
    w = rnd(3, (40, 6), dtype).to(device)
    f = lambda v: (F.q4_linear(v, q, e, 40).t() * w).sum()
    (want,) = torch.autograd.grad(f(x), x)
    torch._dynamo.reset()
    (got,) = torch.autograd.grad(torch.compile(f, backend="aot_eager", fullgraph=True)(x), x)
    assert torch.equal(want, got)


def test_compiled_eager_tier():
    check_compiled("cpu", torch.float32)


def check_traced_outputs(device, dtype):
    """What tracing takes outputs for: shapes, types, strides, for arguments in any order of memory."""
    from torch._subclasses.fake_tensor import FakeTensorMode

    W = rnd(1, (40, 72), dtype).to(device)
    q, e = F.q4_pack_weight(W)
    A, B = rnd(2, (8, 72), dtype).to(device), rnd(3, (40, 8), dtype).to(device)
    n = torch.ones(40, device=device)
    calls = [(F.q4_pack_weight, (W,)), (F.q4_unpack_weight, (q, e, 33, 72, dtype)),
             (F.q4_linear, (rnd(4, (5, 72), dtype).to(device), q, e, 40)),
             (F.q4_linear_backward, (rnd(5, (5, 40), dtype).to(device), q, e, 72)),
             (F.q4_weight_norm, (q, e, A, B, n, 1.5)), (F.q4_weight_norm_backward, (q, e, A, B, n, n, 1.5))]
    turned = lambda a: a.t().contiguous().t() if isinstance(a, torch.Tensor) and a.dim() == 2 else a
    for op, args in calls:
        for call in (args, tuple(turned(a) for a in args)):
            real = op(*call)
            with FakeTensorMode() as mode:
                fake = op(*[mode.from_tensor(a) if isinstance(a, torch.Tensor) else a for a in call])
            for r, f in zip(*(o if isinstance(o, tuple) else (o,) for o in (real, fake))):
                assert (r.shape, r.dtype, r.stride()) == (f.shape, f.dtype, f.stride()), op


def test_traced_outputs_eager():
    check_traced_outputs("cpu", torch.float32)


def check_wrong_layouts(device, dtype):
    q, e = F.q4_pack_weight(torch.zeros(40, 72, device=device, dtype=dtype))
    x = torch.zeros(2, 72, device=device, dtype=dtype)
    for bad in ((x, q[:1], e, 40), (x, q, e[:, :1], 40), (x, q, e, 65), (x, q, e, 32), (x[:, :64], q, e, 40),
                (x, q.to(torch.int32), e, 40), (x, q.reshape(2, -1), e, 40)):
        with pytest.raises((ValueError, binding.DoraError)):
            F.q4_linear(*bad)
    for bad in ((x[:, :65], q, e, 72), (x[:, :40], q, e, 129), (x[:, :40], q, e[:1], 72)):
        with pytest.raises((ValueError, binding.DoraError)):
            F.q4_linear_backward(*bad)
    for rows, cols in ((65, 72), (-1, 72), (40, 129)):
        with pytest.raises((ValueError, binding.DoraError)):
            F.q4_unpack_weight(q, e, rows, cols, dtype)


def test_wrong_layouts_are_refused_eager():
    check_wrong_layouts("cpu", torch.float32)


# ------------------------------------------------------------------ the layer


KINDS = [dict(), dict(detach_norm=False), dict(q8_checkpoint=True), dict(q8_checkpoint=True, detach_norm=False)]


def layer_case(device, dtype, kw, seed=0, in_=200, out=152, r=8):
    torch.manual_seed(seed)
    layer = F.DoRALinear(in_, out, r, dtype=dtype, device=device, q4_weight=True, **kw)
    with torch.no_grad():
        layer.lora_B.normal_(0.0, 0.02)
        layer.magnitude.mul_(1.0 + 0.01 * torch.randn_like(layer.magnitude))
    return layer


def check_layer(device, dtype, kw, tol):
    """Output and gradients against the formulas on the values W0 is held as, in 64 bits."""
    layer = layer_case(device, dtype, kw)
    x = torch.randn(21, 200, device=device).to(dtype).requires_grad_()
    dy = torch.randn(21, 152, device=device).to(dtype)
    y = layer(x)
    got = torch.autograd.grad(y, (x, layer.lora_A, layer.lora_B, layer.magnitude), dy)
    W = F.q4_unpack_weight(*layer._packed_weight(), 152, 200, torch.float32).double()
    leaves = [t.detach().double().requires_grad_() for t in (x, layer.lora_A, layer.lora_B, layer.magnitude)]
    X, A, B, m = leaves
    n = torch.linalg.vector_norm(W + layer.s * B @ A, dim=1)
    n = n.detach() if layer.detach_norm else n
    ref = (m / n) * (X @ W.t() + layer.s * (X @ A.t()) @ B.t())
    want = torch.autograd.grad(ref, leaves, dy.double())
    for g, w in zip((y, *got), (ref, *want)):
        g, w = g.detach().double(), w.detach()
        assert float((g - w).norm()) <= tol * float(w.norm()), float((g - w).norm() / w.norm())


@pytest.mark.parametrize("kw", KINDS)
def test_layer_eager(kw):
    # fp32 all through, but for what is kept in 8 bits: values off by up to 2^-4 of
    # themselves, on the mean below 2^-5, in the gradients of A and m
    check_layer("cpu", torch.float32, kw, 2.0**-5 if kw.get("q8_checkpoint") else 2.0**-16)


def test_layer_starts_out_as_the_frozen_layer():
    torch.manual_seed(0)
    layer = F.DoRALinear(72, 40, 4, dtype=torch.float32, q4_weight=True)
    x = torch.randn(5, 72)
    W = F.q4_unpack_weight(*layer._packed_weight(), 40, 72, torch.float32)
    torch.testing.assert_close(layer(x), x @ W.t(), rtol=1e-5, atol=1e-5)
    assert layer.weight is None and layer.weight_q.dtype == torch.uint8
    half = layer.half()
    assert torch.equal(half.weight_q, layer.weight_q) and half.weight_e.dtype == torch.uint8
    with pytest.raises(ValueError, match="both"):
        F.DoRALinear(8, 8, 2, q4_weight=True, q8_weight=True)
    other = F.DoRALinear(72, 40, 4, dtype=torch.float32, q4_weight=True)
    other.load_state_dict({k: v for k, v in layer.float().state_dict().items() if k != "weight_sqnorm"}, strict=False)
    assert torch.equal(other.weight_q, layer.weight_q)


@pytest.mark.parametrize("dtype,to", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float16)])
@pytest.mark.parametrize("kw", KINDS)
def test_layer_under_autocast(dtype, to, kw):
    check_autocast("cpu", dtype, to, kw)


def check_autocast(device, dtype, to, kw):
    layer = layer_case(device, dtype, kw)
    x = torch.randn(7, 200, device=device, requires_grad=True)
    with torch.autocast(torch.device(device).type, to):
        y = layer(x)
        with torch.no_grad():
            tier = layer(x)
        op = F.q4_linear(x, *layer._packed_weight(), 152)
    assert y.dtype == to and tier.dtype == to and op.dtype == to
    for leaf, g in zip((x, layer.lora_A), torch.autograd.grad(y.float().sum() + op.float().sum(), (x, layer.lora_A))):
        assert g.dtype == leaf.dtype and bool(torch.isfinite(g).all())


# ------------------------------------------------------------------ refusals


def _status(status, want, text):
    assert status == want and text in binding.dora_last_error(), (status, binding.dora_last_error())


@pytest.mark.parametrize("name", ["pack", "unpack"])
def test_pack_refusals(name):
    if name == "pack":
        def fn(W=FAR[0], out=64, in_=128, dt=0, q=FAR[1], e=FAR[2]):
            return LIB.dora_q4_pack_weight(W, out, in_, dt, q, e, None)
    else:
        def fn(W=FAR[0], out=64, in_=128, dt=0, q=FAR[1], e=FAR[2]):
            return LIB.dora_q4_unpack_weight(q, e, out, in_, dt, W, None)
    _status(fn(dt=2), UNSUPPORTED, "dtype")
    _status(fn(out=-1), INVALID, "negative")
    _status(fn(in_=1 << 22), UNSUPPORTED, "beyond")
    _status(fn(out=(1 << 22) - 128, in_=(1 << 22) - 128, W=1 << 60, q=1 << 58, e=1 << 56), UNSUPPORTED, "tiles")
    _status(fn(W=None), INVALID, "NULL")
    _status(fn(W=FAR[0] + 1), INVALID, "aligned")
    _status(fn(q=None), INVALID, "NULL")
    _status(fn(q=FAR[1] + 8), INVALID, "alignment")
    _status(fn(e=FAR[2] + 4), INVALID, "alignment")
    _status(fn(W=FAR[1] + 16), INVALID, "overlaps")
    assert fn(out=0, W=None, q=None) == OK and fn(in_=0, W=None, q=None) == OK


def test_pack_refuses_more_threads_than_a_launch_holds():
    n = 1 << 20  # 2^40 elements, 32 a thread
    _status(LIB.dora_q4_pack_weight(1 << 60, n, n, 0, 1 << 58, 1 << 56, None), UNSUPPORTED, "threads")
    _status(LIB.dora_q4_unpack_weight(1 << 58, 1 << 56, n, n, 0, 1 << 60, None), UNSUPPORTED, "threads")


def test_workspace_is_that_of_the_sizes_whatever_came_before():
    """The plans are kept by their sizes: asked in another order, and in another thread, the answers are the same."""
    sizes = [(T, o, i) for T in (1, 2, 17, 48, 49, 300, 4096) for o in (96, 4096, 5121) for i in (64, 1000, 8192)]

    def ask(order):
        return {(k, s): getattr(LIB, f"dora_q4_linear_{k}workspace_bytes")(*s) for s in order for k in ("", "bwd_")}

    first = ask(sizes)
    assert len(set(first.values())) > 10 and ask(sizes[::-1]) == first
    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        assert all(a == first for a in pool.map(ask, [sizes, sizes[::-1], sizes[::2] + sizes[1::2], sizes]))


@pytest.mark.parametrize("name", ["fwd", "bwd"])
def test_linear_refusals(name):
    fn = getattr(LIB, f"dora_q4_linear_{name}")
    query = LIB.dora_q4_linear_workspace_bytes if name == "fwd" else LIB.dora_q4_linear_bwd_workspace_bytes

    def call(x=FAR[0], q=FAR[1], e=FAR[2], T=200, out=256, in_=4096, dt=0, y=FAR[3], ws=FAR[4], wsb=1 << 39):
        return fn(x, q, e, T, out, in_, dt, y, ws, wsb, None)

    _status(call(dt=2), UNSUPPORTED, "dtype")
    _status(call(T=-1), INVALID, "negative")
    _status(call(out=1 << 22), UNSUPPORTED, "beyond")
    _status(call(T=1 << 31), UNSUPPORTED, "beyond")
    _status(call(y=None), INVALID, "NULL")
    _status(call(y=FAR[3] + 1), INVALID, "alignment")
    _status(call(x=None), INVALID, "rows")
    _status(call(x=FAR[0] + 2), INVALID, "aligned")
    _status(call(q=FAR[1] + 8), INVALID, "packed weight")
    _status(call(e=None), INVALID, "packed weight")
    _status(call(y=FAR[1]), INVALID, "overlaps")
    _status(call(y=FAR[0] + 2), INVALID, "overlaps")
    # rows that are no multiple of 8 elements are copied into the workspace
    T, out, in_ = 200, 251, 4099
    need = query(T, out, in_)
    assert need >= T * (in_ if name == "fwd" else out) * 2
    _status(call(T=T, out=out, in_=in_, wsb=need - 1), INVALID, "workspace of")
    _status(call(T=T, out=out, in_=in_, ws=None), INVALID, "workspace is NULL")
    _status(call(T=T, out=out, in_=in_, ws=FAR[4] + 4), INVALID, "aligned")
    _status(call(T=T, out=out, in_=in_, ws=FAR[3]), INVALID, "overlaps")
    assert call(T=0, x=None, y=None) == OK
    assert call(**({"out": 0} if name == "fwd" else {"in_": 0}), y=None) == OK
    assert query(0, 8, 8) == 0 and query(-1, 8, 8) == 0 and query(8, 1 << 24, 8) == 0


def test_norm_refusals():
    def call(q=FAR[0], e=FAR[1], A=FAR[2], B=FAR[3], c=FAR[4], out=256, in_=512, r=16, dt=0, n=FAR[5], ws=FAR[6],
             wsb=1 << 39):
        return LIB.dora_q4_norm_cached(q, e, A, B, c, out, in_, r, 1.0, dt, n, ws, wsb, None)

    _status(call(dt=2), UNSUPPORTED, "dtype")
    _status(call(out=-1), INVALID, "negative")
    _status(call(r=-8), INVALID, "negative")
    for sizes in ({"r": 0}, {"r": 12}, {"r": 520}, {"in_": 0}, {"in_": 515}, {"in_": 1 << 21}):
        _status(call(**sizes), UNSUPPORTED, "multiples of 8")
        s = {"r": 16, "in_": 512, **sizes}
        assert LIB.dora_q4_norm_workspace_bytes(256, s["in_"], s["r"], 0) == 0
    _status(call(out=1 << 22), UNSUPPORTED, "beyond")
    _status(call(q=None), INVALID, "packed weight")
    _status(call(e=FAR[1] + 4), INVALID, "alignment")
    _status(call(A=None), INVALID, "NULL")
    _status(call(B=FAR[3] + 2), INVALID, "aligned")
    _status(call(c=None), INVALID, "base_sq")
    _status(call(n=FAR[5] + 2), INVALID, "norm_out")
    need = LIB.dora_q4_norm_workspace_bytes(256, 512, 16, 0)
    _status(call(wsb=need - 1), INVALID, "workspace of")
    _status(call(ws=None, wsb=need), INVALID, "workspace is NULL")
    _status(call(ws=FAR[6] + 8), INVALID, "aligned")
    _status(call(n=FAR[4]), INVALID, "overlaps")
    _status(call(ws=FAR[0] - need + 16), INVALID, "overlaps")
    _status(call(n=FAR[6] + 16), INVALID, "overlaps")
    assert call(out=0, q=None) == OK


def test_binding_refuses_other_devices_and_types():
    q, e = F.q4_pack_weight(torch.zeros(4, 200).bfloat16())
    with pytest.raises(ValueError, match="HIP device"):
        binding.dora_q4_pack_weight(torch.zeros(4, 200).bfloat16())
    with pytest.raises(ValueError, match="HIP device"):
        binding.dora_q4_linear_fwd(torch.zeros(4, 200).bfloat16(), q, e, 4)
    with pytest.raises(ValueError, match="HIP device"):
        binding.dora_q4_unpack_weight(q, e, 4, 200, torch.bfloat16)
