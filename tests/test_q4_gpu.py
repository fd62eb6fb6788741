"""The 4-bit weight on the GPU against the fp64 oracle.

Tolerances.  Packed bytes are equal bit for bit (the scaling is exact, and each value
is rounded once), unpacked values exact.  A product y = sum_k a_k b_k of K exact
products of 16-bit operands, rounded once to the output type: each fp32 addition is off
by at most one unit 2^-23 of the running sum (half a unit where it rounds to nearest, a
whole one where it truncates), and that sum is at most the sum of magnitudes.  So
|y - ref| <= eps/2 |ref| (1 + small) + K 2^-23 sum_k |a_k b_k| + half the type's
subnormal step.
"""
import numpy as np
import pytest
import torch

from oracle import dora_oracle as O
from oracle import q4_oracle as Q
from test_q4_cpu import (KINDS, check_autocast, check_compiled, check_layer, check_traced_outputs, check_wrong_layouts,
                         layer_case, rnd, special_weight)

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
SUB = {torch.bfloat16: 2.0**-134, torch.float16: 2.0**-25}


@pytest.fixture(scope="module")
def b():
    from dora_fine_tuning_amd import binding

    return binding


@pytest.fixture(scope="module")
def F():
    from dora_fine_tuning_amd import torch_ops

    return torch_ops


def values(b, q, e, out, in_):
    """The weight's values in fp64 (unpacking is exact, and tested to be)."""
    return b.dora_q4_unpack_weight(q, e, out, in_, torch.bfloat16).double()


def assert_product(got, x, M, what=""):
    """got = x M to the tolerance above (64-bit products on the GPU)."""
    xd = x.to(DEV).double()
    ref, mass = xd @ M, xd.abs() @ M.abs()
    tol = HALF[got.dtype] * (1 + 2.0**-10) * ref.abs() + M.shape[0] * 2.0**-23 * mass + SUB[got.dtype]
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3], ref[bad][:3])


def weight(b, out, in_, dtype, seed=1, scale=0.02, spread=1.0):
    W = rnd(seed, (out, in_), dtype, scale, spread)
    return (*b.dora_q4_pack_weight(W.to(DEV)), W)


# ------------------------------------------------------------------ pack, unpack


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 64), (31, 63), (33, 65), (70, 200), (32, 256), (257, 512), (100, 1032)])
def test_pack_is_the_oracle(b, shape, dtype):
    W = rnd(shape[0] * 7 + shape[1], shape, DT[dtype], spread=6.0)
    rq, re_ = Q.pack(O.as_f64(W))
    for off in (0, 1):  # 16-byte aligned, and not
        buf = torch.empty(W.numel() + off, dtype=W.dtype, device=DEV)
        V = buf[off:].view(shape)
        V.copy_(W)
        q, e = b.dora_q4_pack_weight(V)
        assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(e.cpu().numpy(), re_)
    held = Q.held(O.as_f64(W))
    for dt in DT.values():
        got = b.dora_q4_unpack_weight(q, e, *shape, dt)
        assert np.array_equal(got.double().cpu().numpy(), held, equal_nan=True)
        some = max(1, shape[0] // 2)
        assert torch.equal(b.dora_q4_unpack_weight(q, e, some, shape[1], dt).nan_to_num(), got[:some].nan_to_num())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_pack_special_values(b, dtype):
    W = special_weight(DT[dtype])
    rq, re_ = Q.pack(O.as_f64(W))
    q, e = b.dora_q4_pack_weight(W.to(DEV))
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(e.cpu().numpy(), re_)
    held = Q.held(O.as_f64(W))
    for dt in DT.values():  # from 2^-24 to 6 * 2^13, exact in both
        assert np.array_equal(b.dora_q4_unpack_weight(q, e, *W.shape, dt).double().cpu().numpy(), held, equal_nan=True)


def test_eager_tier_packs_the_same_bytes(F):
    for dt in DT.values():
        W = special_weight(dt)
        for got, want in zip(F.q4_pack_weight(W.to(DEV)), F.q4_pack_weight(W)):
            assert torch.equal(got.cpu(), want)


# ------------------------------------------------------------------ products


TOKENS = [1, 2, 7, 15, 16, 17, 31, 33, 48, 63, 64, 65, 100, 128, 129, 200, 257, 300, 513, 1000]
WEIGHTS = [(1, 1), (5, 7), (40, 72), (33, 100), (65, 129), (152, 200), (264, 1000), (1030, 520), (512, 4096),
           (300, 8192)]


@pytest.mark.parametrize("out,in_", WEIGHTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_forward(b, out, in_, dtype):
    q, e, _ = weight(b, out, in_, DT[dtype])
    M = values(b, q, e, out, in_).t()
    for T in TOKENS:
        x = rnd(T, (T, in_), DT[dtype]).to(DEV)
        assert_product(b.dora_q4_linear_fwd(x, q, e, out), x, M, T)


@pytest.mark.parametrize("out,in_", WEIGHTS + [(8192, 300), (4096, 512)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_backward(b, out, in_, dtype):
    q, e, _ = weight(b, out, in_, DT[dtype])
    M = values(b, q, e, out, in_)
    for T in TOKENS:
        g = rnd(T, (T, out), DT[dtype], spread=2.0).to(DEV)
        assert_product(b.dora_q4_linear_bwd(g, q, e, in_), g, M, T)


@pytest.mark.parametrize("T,out,in_", [(2048, 2048, 2048), (4096, 1024, 4096), (2304, 2816, 1024), (1300, 3000, 2600),
                                       (8192, 512, 512), (700, 8192, 1024), (5000, 640, 1280)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_batches(b, T, out, in_, dtype):
    q, e, _ = weight(b, out, in_, DT[dtype])
    W = values(b, q, e, out, in_)
    x, g = rnd(2, (T, in_), DT[dtype]).to(DEV), rnd(3, (T, out), DT[dtype], spread=2.0).to(DEV)
    assert_product(b.dora_q4_linear_fwd(x, q, e, out), x, W.t())
    assert_product(b.dora_q4_linear_bwd(g, q, e, in_), g, W)


@pytest.mark.parametrize("T", [1, 20, 300])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_whole_range_of_scales(b, T, dtype):
    """Weights from fp16's smallest subnormal to 6 * 2^13 in neighbouring blocks: operands exact in both types."""
    out, in_ = 96, 320
    rng = np.random.default_rng(4)
    W = rng.standard_normal((out, in_)) * np.repeat(np.exp2(rng.integers(-26, 14, (out, in_ // 32))), 32, axis=1)
    W = torch.from_numpy(np.clip(W, -60000, 60000)).to(torch.float16)
    q, e = b.dora_q4_pack_weight(W.to(DEV))
    V = torch.from_numpy(Q.held(O.as_f64(W))).to(DEV)
    x, g = rnd(5, (T, in_), DT[dtype]).to(DEV), rnd(6, (T, out), DT[dtype], 2.0**-6).to(DEV)
    x[:, ::2] *= 2.0**-6  # keeps fp16's results inside its range
    x = x * 2.0**-6
    for got, a, M in ((b.dora_q4_linear_fwd(x, q, e, out), x, V.t()), (b.dora_q4_linear_bwd(g, q, e, in_), g, V)):
        assert bool(torch.isfinite(got).all())
        assert_product(got, a, M)


@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_not_finite(b, T):
    """A NaN or infinity in a row stays in that row's result, a NaN block in its column (its 32 backward)."""
    out, in_ = 72, 136
    W = rnd(1, (out, in_), torch.bfloat16, 0.02)
    q, e = b.dora_q4_pack_weight(W.to(DEV))
    x, g = rnd(2, (T, in_), torch.bfloat16).to(DEV), rnd(3, (T, out), torch.bfloat16).to(DEV)
    clean = b.dora_q4_linear_fwd(x, q, e, out), b.dora_q4_linear_bwd(g, q, e, in_)
    x[T - 1, in_ - 1], g[T - 1, out - 1] = float("nan"), float("inf")
    y, dx = b.dora_q4_linear_fwd(x, q, e, out), b.dora_q4_linear_bwd(g, q, e, in_)
    assert bool(y[T - 1].isnan().all()) and not bool(dx[T - 1].isfinite().any())
    assert torch.equal(y[: T - 1], clean[0][: T - 1]) and torch.equal(dx[: T - 1], clean[1][: T - 1])
    W[40, 33] = float("nan")
    q, e = b.dora_q4_pack_weight(W.to(DEV))
    y = b.dora_q4_linear_fwd(rnd(2, (T, in_), torch.bfloat16).to(DEV), q, e, out)
    assert bool(y[:, 40].isnan().all()) and int(y.isnan().sum()) == T
    dx = b.dora_q4_linear_bwd(rnd(3, (T, out), torch.bfloat16).to(DEV), q, e, in_)
    assert bool(dx[:, 32:64].isnan().all()) and int(dx.isnan().sum()) == 32 * T


def test_columns_past_the_weight_read_nothing(b):
    """The row behind a short row is not part of it: its values may be anything."""
    for in_, out in ((40, 64), (72, 64), (136, 96), (200, 40)):
        q, e, _ = weight(b, out, in_, torch.bfloat16)
        W = values(b, q, e, out, in_)
        for T in (3, 70, 300):
            x, g = rnd(2, (T, in_), torch.bfloat16).to(DEV), rnd(3, (T, out), torch.bfloat16).to(DEV)
            x[1::2], g[1::2] = float("nan"), float("inf")
            y, dx = b.dora_q4_linear_fwd(x, q, e, out), b.dora_q4_linear_bwd(g, q, e, in_)
            assert_product(y[::2], x[::2], W.t(), (T, in_))
            assert_product(dx[::2], g[::2], W, (T, out))


def test_results_repeat_bit_for_bit(b):
    for T, out, in_ in ((1, 512, 4096), (37, 512, 4096), (300, 4096, 2048), (2304, 2816, 1024)):
        q, e, _ = weight(b, out, in_, torch.bfloat16)
        x, g = rnd(2, (T, in_), torch.bfloat16).to(DEV), rnd(3, (T, out), torch.bfloat16).to(DEV)
        y, dx = b.dora_q4_linear_fwd(x, q, e, out), b.dora_q4_linear_bwd(g, q, e, in_)
        for _ in range(5):
            assert torch.equal(b.dora_q4_linear_fwd(x, q, e, out), y)
            assert torch.equal(b.dora_q4_linear_bwd(g, q, e, in_), dx)


def test_outputs_write_nothing_else(b):
    """Bytes around y, and a workspace just as large as asked for."""
    from dora_fine_tuning_amd.binding import LIB, _ptr, _raw_stream

    for T, out, in_ in ((1, 40, 72), (5, 41, 73), (37, 33, 200), (300, 250, 1000), (130, 129, 4097), (500, 72, 8200)):
        for name, N, K in (("fwd", out, in_), ("bwd", in_, out)):
            q, e, _ = weight(b, out, in_, torch.bfloat16)
            x = rnd(1, (T, K), torch.bfloat16).to(DEV)
            want = b.dora_q4_linear_fwd(x, q, e, out) if name == "fwd" else b.dora_q4_linear_bwd(x, q, e, in_)
            query = LIB.dora_q4_linear_workspace_bytes if name == "fwd" else LIB.dora_q4_linear_bwd_workspace_bytes
            need = int(query(T, out, in_))
            ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
            for off in (8, 9):
                buf = torch.full((T * N + 32,), 7.0, dtype=torch.bfloat16, device=DEV)
                y = buf[off : off + T * N]
                fn = getattr(LIB, f"dora_q4_linear_{name}")
                st = fn(_ptr(x), _ptr(q), _ptr(e), T, out, in_, 0, _ptr(y), _ptr(ws), need, _raw_stream(DEV))
                assert st == 0, b.dora_last_error()
                assert torch.equal(y.view(T, N), want), (name, T, out, in_, off)
                assert bool((buf[:off] == 7).all()) and bool((buf[off + T * N :] == 7).all())
                assert bool((ws[need:] == 0x5A).all())


def test_rows_past_2_32_bytes(b):
    T, out, in_ = 300_000, 40, 8192
    q, e, _ = weight(b, out, in_, torch.bfloat16)
    W = values(b, q, e, out, in_)
    x = torch.randn((T, in_), device=DEV, dtype=torch.bfloat16)  # 4.9 GB
    y = b.dora_q4_linear_fwd(x, q, e, out)
    for i in range(0, T, 50_000):
        assert_product(y[i : i + 50_000], x[i : i + 50_000], W.t(), i)
    dx = b.dora_q4_linear_bwd(y, q, e, in_)
    for i in range(0, T, 50_000):
        assert_product(dx[i : i + 50_000], y[i : i + 50_000], W, i)


def test_weight_past_2_32_bytes(b):
    """9.8e9 values, 4.9e9 bytes: first, middle and last rows and columns."""
    out, in_ = 300_000, 32_768
    qs, es = b.q4_weight_shapes(out, in_)
    q = torch.randint(0, 256, qs, dtype=torch.uint8, device=DEV)
    e = torch.randint(118, 123, es, dtype=torch.uint8, device=DEV)
    x = rnd(1, (3, in_), torch.bfloat16).to(DEV)
    y = b.dora_q4_linear_fwd(x, q, e, out)
    for r in (0, 149_984, 299_968):
        rows = slice(r, min(r + 32, out))
        W = values(b, q[r // 32 : r // 32 + 1].contiguous(), e[r // 32 : r // 32 + 1].contiguous(), rows.stop - r, in_)
        assert_product(y[:, rows], x, W.t(), r)
    g = torch.zeros((2, out), dtype=torch.bfloat16, device=DEV)
    g[0, -40:], g[1, 150_000:150_040] = 1.0, 0.5
    dx = b.dora_q4_linear_bwd(g, q, e, in_)
    for t, r in ((0, 299_936), (1, 149_984)):
        n = min(96, out - r)
        W = values(b, q[r // 32 : r // 32 + 3].contiguous(), e[r // 32 : r // 32 + 3].contiguous(), n, in_)
        assert_product(dx[t : t + 1], g[t : t + 1, r : r + n], W, r)


# ------------------------------------------------------------------ as it is used


def test_strides_slices_and_streams(F, b):
    out, in_ = 152, 200
    q, e, _ = weight(b, out, in_, torch.bfloat16)
    W = values(b, q, e, out, in_)
    wide = torch.randn((30, 2 * in_ + 1), device=DEV).bfloat16()
    for x in (wide[:, 1 : 1 + in_], wide.t()[:in_, :].t(), wide[::3, :in_],
              wide.reshape(-1)[1 : 1 + 20 * in_].view(20, in_), wide[:1, :in_].expand(6, in_)):
        assert_product(F.q4_linear(x, q, e, out), x, W.t())
    s = torch.cuda.Stream()
    x = wide[:, :in_].contiguous()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = F.q4_linear(x, q, e, out)
        dx = F.q4_linear_backward(y, q, e, in_)
    torch.cuda.current_stream().wait_stream(s)
    assert_product(y, x, W.t())
    assert_product(dx, y, W)


def test_captured_and_replayed(F, b):
    """Two captured graphs and eager calls between their replays, at sizes with and without a workspace."""
    cases = []
    for T, out, in_ in ((1, 512, 4096), (37, 500, 1001), (300, 4096, 512)):
        q, e, _ = weight(b, out, in_, torch.bfloat16)
        x = torch.randn((T, in_), device=DEV).bfloat16()
        run = lambda x=x, q=q, e=e, out=out, in_=in_: F.q4_linear_backward(F.q4_linear(x, q, e, out), q, e, in_)
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = run()
        cases.append((g, x, y, run))
    for i in range(4):
        for g, x, y, run in cases:
            x.copy_(torch.randn_like(x))
            g.replay()
            assert torch.equal(y, run()), i


def test_training_captured(F, b):
    """(With no eager graph of x alive: torch would run x's end of the backward on that graph's stream.)"""
    q, e, _ = weight(b, 152, 200, torch.bfloat16)
    x = torch.randn((33, 200), device=DEV).bfloat16().requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step = lambda: torch.autograd.grad(F.q4_linear(x, q, e, 152), x, dy)[0]
    dy = torch.randn((33, 152), device=DEV).bfloat16()
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dx = step()
    for _ in range(3):
        dy.copy_(torch.randn_like(dy))
        g.replay()
        assert torch.equal(dx, F.q4_linear_backward(dy, q, e, 200))
        (again,) = torch.autograd.grad(F.q4_linear(x, q, e, 152), x, dy)
        assert torch.equal(again, dx)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gradient(F, b, dtype):
    out, in_ = 152, 200
    q, e, _ = weight(b, out, in_, DT[dtype])
    x = rnd(1, (40, in_), DT[dtype]).to(DEV).requires_grad_()
    dy = rnd(2, (40, out), DT[dtype]).to(DEV)
    (dx,) = torch.autograd.grad(F.q4_linear(x, q, e, out), x, dy)
    assert_product(dx, dy, values(b, q, e, out, in_))
    (dx,) = torch.autograd.grad(F.q4_linear(x, q, e, out).sum(), x)  # dy of stride 0
    assert_product(dx, torch.ones_like(dy), values(b, q, e, out, in_))


def test_eager_types_on_the_gpu(F):
    q, e = F.q4_pack_weight(torch.randn((40, 72), device=DEV))
    x = torch.randn((5, 72), device=DEV)
    W = F.q4_unpack_weight(q, e, 40, 72, torch.float32)
    torch.testing.assert_close(F.q4_linear(x, q, e, 40), x @ W.t(), rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("T,out,in_", [(0, 40, 72), (5, 0, 72), (5, 40, 0), (0, 0, 0)])
def test_empty(F, T, out, in_):
    q, e = F.q4_pack_weight(torch.zeros((out, in_), device=DEV, dtype=torch.bfloat16))
    y = F.q4_linear(torch.ones((T, in_), device=DEV, dtype=torch.bfloat16), q, e, out)
    dx = F.q4_linear_backward(torch.ones((T, out), device=DEV, dtype=torch.bfloat16), q, e, in_)
    assert y.shape == (T, out) and dx.shape == (T, in_) and not bool(y.any()) and not bool(dx.any())


@pytest.mark.parametrize("kw", KINDS)
def test_layer(kw):
    # bf16: each of the up to six roundings on a path is off by 2^-9 of its value on
    # the root mean square; what is kept in 8 bits by up to 2^-4, below 2^-5 on the mean
    check_layer(DEV, torch.bfloat16, kw, 2.0**-5 if kw.get("q8_checkpoint") else 2.0**-6)


def test_layer_norm_is_that_of_the_held_weight(F):
    layer = layer_case(DEV, torch.bfloat16, {}, in_=520, out=4100, r=16)  # three slabs of rows
    W = F.q4_unpack_weight(*layer._packed_weight(), 4100, 520, torch.float32).double()
    n = torch.linalg.vector_norm(W + layer.s * layer.lora_B.double() @ layer.lora_A.double(), dim=1)
    assert bool(((layer.weight_norm().double() - n).abs() <= 1e-5 * n).all())
    fresh = F.DoRALinear(520, 4100, 16, device=DEV, q4_weight=True)
    assert torch.equal(fresh.magnitude, fresh.weight_norm())  # g = 1 exactly


@pytest.mark.parametrize("dtype,to", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float16)])
@pytest.mark.parametrize("kw", KINDS)
def test_layer_under_autocast(dtype, to, kw):
    check_autocast(DEV, dtype, to, kw)


def test_compiled():
    check_compiled(DEV, torch.bfloat16)


def test_traced_outputs():
    check_traced_outputs(DEV, torch.bfloat16)


def test_wrong_layouts_are_refused():
    check_wrong_layouts(DEV, torch.bfloat16)
