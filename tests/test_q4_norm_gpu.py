"""The norm of a packed 4-bit weight on the GPU against the fp64 oracle.

Tolerance: the norm's own (relative 1e-5, or 2^-16 of the term mass where the terms
cancel): products exact in fp32, sums in fp32, (s/2) A A^T as two 16-bit values.
"""
import pytest
import torch

import parity_util as PU
from oracle import dora_oracle as O
from test_q4_cpu import rnd

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def b():
    from dora_fine_tuning_amd import binding

    return binding


@pytest.fixture(scope="module")
def F():
    from dora_fine_tuning_amd import torch_ops

    return torch_ops


def case(b, out, in_, r, dtype, seed=1, scale=0.05):
    q, e = b.dora_q4_pack_weight(rnd(seed, (out, in_), dtype, 0.02).to(DEV))
    W = b.dora_q4_unpack_weight(q, e, out, in_, torch.bfloat16)
    A, B = rnd(seed + 1, (r, in_), dtype, 0.05).to(DEV), rnd(seed + 2, (out, r), dtype, scale).to(DEV)
    return q, e, W, A, B, b.dora_row_sqnorm(W)


def check(got, W, A, B, c, s, what):
    got, W, A, B, c = (t.double().cpu().numpy() for t in (got, W, A, B, c))
    PU.assert_norm(got, O.weight_norm_cached(c, W, A, B, s), PU.norm_term_mass(W, A, B, s), what)


# every kernel of the product (few rows with one to three token tiles, the tiles), one
# range and more, ranks that end inside a step of 32 and a tile of 16
RANKS = [8, 16, 24, 32, 40, 48, 56, 64, 96, 128, 200, 264, 384, 512]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("r", RANKS)
@pytest.mark.parametrize("out,in_", [(1, 8), (33, 72), (300, 520), (1000, 2056), (96, 8200)])
def test_norm(b, out, in_, r, dtype):
    q, e, W, A, B, c = case(b, out, in_, r, DT[dtype])
    check(b.dora_q4_norm_cached(q, e, A, B, c, 0.7), W, A, B, c, float(torch.tensor(0.7)), (out, in_, r))


@pytest.mark.parametrize("out,in_,r", [(4096, 4096, 16), (8192, 1024, 384), (20000, 512, 512), (5120, 2048, 64)])
def test_norm_of_large_weights(b, out, in_, r):
    """More tiles than the card holds workgroups among them."""
    q, e, W, A, B, c = case(b, out, in_, r, torch.bfloat16)
    got = b.dora_q4_norm_cached(q, e, A, B, c, 2.0)
    check(got, W, A, B, c, 2.0, (out, in_, r))
    for _ in range(3):
        assert torch.equal(b.dora_q4_norm_cached(q, e, A, B, c, 2.0), got)


# sizes at which each kernel of the product is the one taken, whole and in ranges, and one
# whose product would have whole rounds with ranges behind them (all whole here)
EVERY = [(512, 512, 8), (1024, 8192, 16), (512, 512, 24), (1024, 8192, 24), (512, 512, 40), (1024, 8192, 48),
         (12000, 2000, 16), (12000, 2000, 24), (4096, 4096, 32), (12000, 2000, 40), (4096, 4096, 48),
         (27648, 5120, 16), (8192, 8192, 16), (27648, 5120, 32), (8192, 8192, 32), (27648, 5120, 384),
         (5120, 27648, 264), (27648, 5120, 200), (8192, 8192, 200), (27648, 5120, 264), (512, 512, 64),
         (1024, 8192, 128), (8192, 1024, 264), (4096, 4096, 192), (27648, 5120, 512)]


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("out,in_,r", EVERY)
def test_norm_by_every_kernel(b, out, in_, r, odd):
    """Against 64 bits on the GPU; |B A| is too small beside W for the terms to cancel."""
    out -= 5 * odd
    g = torch.Generator(device=DEV)
    g.manual_seed(out + r)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV).bfloat16()
    q, e = b.dora_q4_pack_weight(rand(out, in_) * 0.02)
    W = b.dora_q4_unpack_weight(q, e, out, in_, torch.bfloat16)
    A, B, c = rand(r, in_) * 0.02, rand(out, r) * 0.02, b.dora_row_sqnorm(W)
    got = b.dora_q4_norm_cached(q, e, A, B, c, 2.0).double()
    V = B.double() @ A.double()
    n = (c.double() + (4.0 * W.double() * V + 4.0 * V * V).sum(dim=1)).sqrt()
    assert bool(((got - n).abs() <= 1e-5 * n).all()), (got / n - 1).abs().max()


@pytest.mark.parametrize("r", [16, 64])
def test_cancelling_rows(b, r):
    """c so small that the sum is negative (0 then), and rows whose terms nearly cancel."""
    q, e, W, A, B, c = case(b, 300, 520, r, torch.bfloat16, scale=0.3)
    check(b.dora_q4_norm_cached(q, e, A, B, c * 0.25, -0.5), W, A, B, c * 0.25, -0.5, r)
    assert not bool(b.dora_q4_norm_cached(q, e, A, B, c * 0 - 1e4, -0.5).any())


def test_zero_adapter_is_the_cache(b):
    q, e, W, A, B, c = case(b, 130, 200, 16, torch.float16)
    assert torch.equal(b.dora_q4_norm_cached(q, e, A, torch.zeros_like(B), c, 3.0), c.double().sqrt().float())


def test_not_finite(b):
    """A block of W that is not finite touches its row alone, a NaN in B its own; both end as the 16-bit norm's."""
    out, in_, r = 70, 264, 24
    W = rnd(1, (out, in_), torch.bfloat16, 0.02)
    W[37, 100] = float("inf")
    q, e = b.dora_q4_pack_weight(W.to(DEV))
    held = b.dora_q4_unpack_weight(q, e, out, in_, torch.bfloat16)
    A, B = rnd(2, (r, in_), torch.bfloat16, 0.05).to(DEV), rnd(3, (out, r), torch.bfloat16, 0.05).to(DEV)
    B[5, 3] = float("nan")
    c = torch.rand(out, device=DEV) + 1
    got, ref = b.dora_q4_norm_cached(q, e, A, B, c, 1.0), b.dora_norm_factored_cached(held, A, B, c, 1.0)
    assert bool(torch.isclose(got, ref, rtol=2e-5, atol=0).all()) and bool(got.isfinite().all())
    assert got[[5, 37]].tolist() == [0.0, 0.0] and int((got == 0).sum()) == 2


def test_operator_streams_slices_and_capture(F, b):
    out, in_, r, s = 300, 1032, 24, 0.5
    q, e, W, A, B, c = case(b, out, in_, r, torch.bfloat16)
    wide_a, wide_b = torch.randn((r, in_ + 1), device=DEV).bfloat16(), torch.randn((r, out), device=DEV).bfloat16()
    A2, B2 = wide_a[:, 1:], wide_b.t() * 0.05  # rows off their alignment, columns outermost
    check(F.q4_weight_norm(q, e, A2, B2, c, s), W, A2, B2, c, s, "strides")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        n = F.q4_weight_norm(q, e, A, B, c, s)
    torch.cuda.current_stream().wait_stream(st)
    check(n, W, A, B, c, s, "stream")
    graphs = []
    for rr in (24, 8):  # two graphs, with eager calls between their replays
        a, bb = A[:rr].clone(), B[:, :rr].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            n = F.q4_weight_norm(q, e, a, bb, c, s)
        graphs.append((g, a, bb, n))
    for i in range(4):
        for g, a, bb, n in graphs:
            a.copy_(torch.randn_like(a) * 0.05)
            g.replay()
            assert torch.equal(n, F.q4_weight_norm(q, e, a, bb, c, s)), i
            check(n, W, a, bb, c, s, i)


@pytest.mark.parametrize("out,in_,r", [(70, 200, 0), (70, 200, 12), (70, 203, 8), (2100, 64, 520)])
def test_sizes_that_go_by_unpacked_rows(F, b, out, in_, r):
    q, e, W, A, B, c = case(b, out, in_, r, torch.bfloat16)
    check(F.q4_weight_norm(q, e, A, B, c, 0.5), W, A, B, c, 0.5, (out, in_, r))


def test_gradients_are_those_of_the_unpacked_weight(F, b):
    q, e, W, A, B, c = case(b, 300, 520, 16, torch.bfloat16)
    d = torch.randn(300, device=DEV)
    grads = []
    for f in (lambda *ab: F.q4_weight_norm(q, e, *ab, c, 0.5), lambda *ab: F.weight_norm_cached(W, *ab, c, 0.5)):
        a, bb = A.clone().requires_grad_(), B.clone().requires_grad_()
        f(a, bb).backward(d)
        grads.append((a.grad.float(), bb.grad.float()))
    # both round once to bf16 (half a step 2^-8 each), from sums of 300 to 520 terms of which each
    # is off by the norm's 2e-5: some sqrt(520) * 2e-5 < 2^-11 of a sum's usual size
    for x, y in zip(*grads):
        assert bool(((x - y).abs() <= 2.0**-7 * y.abs() + 2.0**-8 * y.abs().mean()).all())
