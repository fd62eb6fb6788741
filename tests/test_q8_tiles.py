"""The products where a workgroup takes several units of work in turn, and over
long contractions.

Two bounds hold at once.  Per element, the one of test_q8_gpu: half a step of the
output type, K 2^-23 of the sum of magnitudes for the fp32 sums, and 7 2^-13 of the
largest product of every eight steps for the cut inside the instruction.  It grows
with K: at 27648 it is 0.4 of the output's own size, and a stage left out (1/216
of the sum) passes.  So, per block of 64 x 64 outputs, the norm of the error: the
cut takes each of a group's seven other products towards zero by less than u =
2^-13 max |a| max |b|, wherever in [0, u) its lower bits happen to lie, so with
operands of random sign their errors are uncorrelated with mean square u^2 / 3 at
most, and

    E |err|^2 <= sum over outputs and groups of 7/3 u^2.

A block has at most 4096 outputs, whose mean square scatters by a few per cent
(fewer rows or columns: more), so its root is taken 1.5 times; the fp32 sums,
of K/8 additions each off by at most 2^-23 of a running sum that is as large as
the output at its end and smaller before, add sqrt(K/8) 2^-23 of the norm, and the
rounding half a step of it.  A stage of 128 steps left out of K is sqrt(128/K) of
the norm: 6.8e-2 at 27648, against bounds of 4e-3 (bf16) and 7e-4 (fp16)."""
import numpy as np
import pytest
import torch

from dora_fine_tuning_amd import binding as b

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {"bf16": 2.0**-8, "fp16": 2.0**-11}
SUB = {"bf16": 2.0**-134, "fp16": 2.0**-25}
STEP = 64


def block_norms(sq):
    """Square roots of the sums over 64 x 64 blocks of non-negative values."""
    T, N = sq.shape
    p = torch.nn.functional.pad(sq, (0, -N % STEP, 0, -T % STEP))
    return p.reshape(p.shape[0] // STEP, STEP, -1, STEP).sum(dim=(1, 3)).sqrt()


def groups(x, dim):
    """Largest magnitude of every eight consecutive contraction steps."""
    pad = -x.shape[dim] % 8
    x = torch.nn.functional.pad(x.abs(), (0, pad) if dim == 1 else (0, 0, 0, pad))
    return (x.reshape(x.shape[0], -1, 8).amax(2) if dim == 1 else x.reshape(-1, 8, x.shape[1]).amax(1))


def accepts(y, X, M, dtype):
    """Whether y [T x N] is X [T x K] M [K x N] (fp64) within both bounds."""
    K = X.shape[1]
    ref = X @ M
    gx, gm = groups(X, 1), groups(M, 0)
    tol = HALF[dtype] * (1 + 2.0**-10) * ref.abs() + SUB[dtype] + K * 2.0**-23 * (X.abs() @ M.abs())
    err = (y.double() - ref).abs()
    if not torch.all(err <= tol + 7 * 2.0**-13 * (gx @ gm)):
        return False
    cut = block_norms(7 / 3 * 2.0**-26 * ((gx * gx) @ (gm * gm)))
    norm = block_norms(ref * ref)
    return bool(torch.all(block_norms(err * err) <= 1.5 * cut + (HALF[dtype] + (K / 8) ** 0.5 * 2.0**-23) * norm))


def operands(device, T, N, K, trans, dtype, seed=11):
    """Packed (x, W), and in fp64 the values they hold: X [T x K], M [K x N]."""
    from dora_fine_tuning_amd import torch_ops as F

    g = torch.Generator(device=device).manual_seed(seed)
    out, in_ = (K, N) if trans else (N, K)
    W = (torch.randn(out, in_, generator=g, device=device) * 0.02).to(DT[dtype])
    x = torch.randn(T, K, generator=g, device=device) * torch.exp2(torch.randn(T, 1, generator=g, device=device))
    Wp, xp = F.q8_pack_weight(W), F.q8_pack(x.to(DT[dtype]))
    # bf16 holds every unpacked value exactly
    M = F.q8_unpack_weight(*Wp, out, in_, torch.bfloat16).double()
    return xp, Wp, F.q8_unpack(*xp, K, torch.bfloat16).double(), M if trans else M.t().contiguous()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_the_bounds_find_a_lost_stage(dtype):
    """On the CPU, with the mistake planted in the sum that stands for the kernel."""
    _, _, X, M = operands("cpu", 64, 128, 27648, False, dtype)
    y = X @ M
    assert accepts(y.to(DT[dtype]), X, M, dtype)
    for stage in (0, 100, 215):
        at = slice(128 * stage, 128 * stage + 128)
        assert not accepts((y - X[:, at] @ M[at]).to(DT[dtype]), X, M, dtype)
    one = y.clone()  # one block of one tile alone
    one[:, 64:] -= X[:, 128:256] @ M[128:256, 64:]
    assert not accepts(one.to(DT[dtype]), X, M, dtype)
    moved = y.clone()
    moved[[3, 4]] = moved[[4, 3]]
    assert not accepts(moved.to(DT[dtype]), X, M, dtype)


def run(T, N, K, trans, dtype):
    xp, Wp, X, M = operands("cuda:0", T, N, K, trans, dtype)
    f = b.dora_q8_linear_bwd if trans else b.dora_q8_linear_fwd
    y = f(*xp, *Wp, *((K, N) if trans else (N, K)), DT[dtype])
    assert accepts(y, X, M, dtype)
    assert torch.equal(y, f(*xp, *Wp, *((K, N) if trans else (N, K)), DT[dtype]))


def workspace(T, N, K, trans):
    q = b.LIB.dora_q8_linear_bwd_workspace_bytes if trans else b.LIB.dora_q8_linear_workspace_bytes
    return int(q(T, *((K, N) if trans else (N, K))))


# (direction, T, N, K, tile rows, tile columns): more tiles than CUs, and the ones behind the
# last full round split over the contraction
MIXED = [
    (False, 1005, 16480, 1277, 256, 256), (False, 2304, 8450, 4096, 256, 256), (False, 2050, 8320, 8192, 256, 256),
    (False, 1453, 5447, 2440, 256, 128), (False, 261, 16439, 2816, 192, 128), (False, 203, 16653, 4488, 128, 128),
    (True, 4352, 4096, 4096, 256, 256), (True, 2600, 8192, 8192, 256, 256), (True, 403, 16490, 2688, 256, 128),
    (True, 278, 16392, 2312, 192, 128), (True, 207, 16386, 4221, 128, 128),
]
# more than 256 tiles of any size, too few stages to split, rows that are not multiples of 16 bytes
ROUNDS = [(t, *s) for t in (False, True) for s in ((4353, 4099, 890), (700, 27643, 650), (8200, 4097, 520))]


@pytest.mark.parametrize("trans,T,N,K,bm,bn", MIXED)
def test_mixed_sizes_are_mixed(trans, T, N, K, bm, bn):
    tiles = -(-T // bm) * -(-N // bn)
    ranges, rest = divmod(workspace(T, N, K, trans), (tiles % 256) * bm * bn * 4)
    assert tiles > 256 and rest == 0 and 2 <= ranges <= 16


@pytest.mark.parametrize("trans,T,N,K", ROUNDS)
def test_round_sizes_are_rounds(trans, T, N, K):
    assert -(-T // 256) * -(-N // 256) > 256 and N % 8 and workspace(T, N, K, trans) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("trans,T,N,K,bm,bn", MIXED)
def test_whole_tiles_then_split_ones(trans, T, N, K, bm, bn, dtype):
    run(T, N, K, trans, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("trans,T,N,K", ROUNDS)
def test_rounds_of_tiles_with_single_stores(trans, T, N, K, dtype):
    run(T, N, K, trans, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("T,N", [(1, 5120), (8, 1024), (37, 5120), (300, 2050), (512, 5120)])
def test_long_contraction(T, N, trans, dtype):
    run(T, N, 27648, trans, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("trans", [False, True])
def test_every_row_of_an_output_past_32_bits(trans):
    """Rows that repeat every 64, one stage: each sum is the same four matrix
    instructions in any tile, so all rows equal the first 64, bit for bit."""
    T, N, K = 290000, 8192, 128  # 4.75e9 bytes
    xp, Wp, X, M = operands("cuda:0", 64, N, K, trans, "bf16")
    f = b.dora_q8_linear_bwd if trans else b.dora_q8_linear_fwd
    size = (K, N) if trans else (N, K)
    few = f(*xp, *Wp, *size, torch.bfloat16)
    assert accepts(few, X, M, "bf16")
    q = xp[0].view(torch.uint8).repeat(-(-T // 64), 1)[:T].contiguous().view(torch.float8_e4m3fn)
    e = xp[1].repeat(-(-T // 64), 1)[:T].contiguous()
    y = f(q, e, *Wp, *size, torch.bfloat16)
    assert torch.equal(y[: T // 64 * 64].view(-1, 64, N), few.expand(T // 64, 64, N))
    assert torch.equal(y[T // 64 * 64:], few[: T % 64])
