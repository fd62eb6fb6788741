"""Products with a 4-bit weight whose sums are exact in fp32, so that a result is right
only bit for bit, however long the contraction.

The weight's values are ±{0, 0.5, 1, 1.5, 2, 3, 4, 6} times 2^-1, 1 or 2 a block, which
blocks hold as they are (scaled by a power of two so that the largest is 4 or 6 they
stay on the same list).  The rows are whole numbers from -2 to 2.  Every partial sum, in
whatever order, is then a multiple of 2^-2 of magnitude 24 K at most, and fp32 holds it
while 24 K * 2^2 < 2^24: up to K = 174762.  What is left is one rounding to the type.
"""
import torch

LONGEST = 174762


def weight(out, in_, device, seed=0):
    """Values in fp64."""
    g = torch.Generator(device=device)
    g.manual_seed(seed * 7919 + out * 31 + in_)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device, dtype=torch.float64)
    W = torch.cat((grid, -grid))[torch.randint(0, 16, (out, in_), generator=g, device=device)]
    scales = torch.randint(-1, 2, (out, -(-in_ // 32)), generator=g, device=device).double().exp2()
    return W * scales.repeat_interleave(32, dim=1)[:, :in_]


def rows(T, K, device, seed=1):
    assert K <= LONGEST
    g = torch.Generator(device=device)
    g.manual_seed(seed * 104729 + T * 31 + K)
    return torch.randint(-2, 3, (T, K), generator=g, device=device).double()


def assert_exact(got, x, M, what=""):
    """got is x M (fp64, exact), rounded once."""
    ref = (x @ M).to(got.dtype)
    bad = got != ref
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3], ref[bad][:3])
