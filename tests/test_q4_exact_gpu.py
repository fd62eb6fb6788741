"""The 4-bit products bit for bit, on operands whose sums are exact (q4_exact): the sizes
of test_q4_kernels_gpu and others with long contractions, whose ranges, tails and ring
run over hundreds of stages.  A tolerance that grows with the contraction does not see a
column that is left out there; these do (test_q4_exact_cpu)."""
import pytest
import torch

from q4_exact import assert_exact, rows, weight
from test_q4_kernels_gpu import BACKWARD, FORWARD

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
# contractions that end one column, one block or one stage past a whole step, and up to 2^17
LONG = [(T, n, K) for T in (1, 16, 33, 65, 300) for n, K in ((65, 27647), (64, 27681), (128, 27713), (33, 131072))]


@pytest.fixture(scope="module")
def b():
    from dora_fine_tuning_amd import binding

    return binding


def check(b, T, out, in_, trans, dtype):
    W = weight(out, in_, DEV)
    q, e = b.dora_q4_pack_weight(W.to(dtype))
    x = rows(T, out if trans else in_, DEV)
    y = b.dora_q4_linear_bwd(x.to(dtype), q, e, in_) if trans else b.dora_q4_linear_fwd(x.to(dtype), q, e, out)
    assert_exact(y, x, W if trans else W.t(), (T, out, in_))


@pytest.mark.parametrize("odd,dtype", [(False, "bf16"), (True, "fp16")])
@pytest.mark.parametrize("T,out,in_", FORWARD)
def test_forward(b, T, out, in_, odd, dtype):
    if odd:
        T, out, in_ = max(1, T - T // 20), out - 5, in_ - 3
    check(b, T, out, in_, False, DT[dtype])


@pytest.mark.parametrize("odd,dtype", [(False, "fp16"), (True, "bf16")])
@pytest.mark.parametrize("T,out,in_", BACKWARD)
def test_backward(b, T, out, in_, odd, dtype):
    if odd:
        T, out, in_ = max(1, T - T // 20), out - 3, in_ - 5
    check(b, T, out, in_, True, DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,n,K", LONG)
def test_long_contractions(b, T, n, K, dtype):
    check(b, T, n, K, False, DT[dtype])
    check(b, T, K, n, True, DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_contraction_length(b, dtype):
    """Each K up to four stages and around more, by few rows and by tiles."""
    for K in [*range(1, 258), 511, 512, 513, 767, 1023, 1025, 4095, 4097]:
        for T in (3, 70):
            check(b, T, 40, K, False, DT[dtype])
            check(b, T, K, 40, True, DT[dtype])
