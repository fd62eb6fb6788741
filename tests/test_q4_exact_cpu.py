"""The comparison of test_q4_exact_gpu sees lost work: on the CPU, with the mistakes in
a plain product."""
import pytest
import torch

from dora_fine_tuning_amd import binding  # noqa: F401  (the library is there)
from q4_exact import LONGEST, assert_exact, rows, weight

F = pytest.importorskip("dora_fine_tuning_amd.torch_ops")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_operands_are_held_as_they_are(dtype):
    W = weight(70, 200, "cpu")
    q, e = F.q4_pack_weight(W.to(dtype))
    assert torch.equal(F.q4_unpack_weight(q, e, 70, 200, dtype).double(), W)
    x = rows(9, 200, "cpu")
    assert torch.equal(x.to(dtype).double(), x)
    assert_exact(F.q4_linear(x.to(dtype), q, e, 70), x, W.t())


def test_sums_are_exact():
    """The bound of the docstring: a sum of the largest magnitudes, one by one in fp32."""
    assert 24 * LONGEST * 4 < 2**24 <= 24 * (LONGEST + 1) * 4
    x, W = rows(1, 20000, "cpu").abs() + 1, weight(1, 20000, "cpu").abs()
    s = torch.zeros((), dtype=torch.float32)
    for t in torch.unbind((x * W).float().flatten()):
        s = s + t
    assert float(s) == float((x * W).sum())


@pytest.mark.parametrize("K", [20000, 27648])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lost", [64, 32, 1])
def test_lost_work_is_seen(K, dtype, lost):
    """A stage, a block or a single column that is left out or taken twice, in one row tile of one token tile."""
    x, M = rows(16, K, "cpu"), weight(32, K, "cpu").t()
    y = x @ M
    assert_exact(y.float().to(dtype), x, M)
    at = K // 2 - lost
    part = x[:, at : at + lost] @ M[at : at + lost]
    for wrong in (y - part, y + part):
        with pytest.raises(AssertionError):
            assert_exact(wrong.float().to(dtype), x, M)
