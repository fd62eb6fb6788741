"""Every kernel of the 4-bit products: sizes at which each of them is the one that a
call takes, as far as the choice goes by size: few rows in groups of one, two or four
row tiles and of one to three token tiles, whole and in ranges of the contraction;
tiles of 64 x 128, 48, 64, 96 and 128 x 256, in whole rounds, in one round that is not
full, in ranges, and in whole rounds with ranges behind them.  Each size as it is and
with odd numbers of rows and columns, in both types (tolerances in test_q4_gpu)."""
import pytest
import torch

from test_q4_gpu import DEV, DT, assert_product, values

pytestmark = pytest.mark.gpu

FORWARD = [(1, 512, 512), (1, 1024, 8192), (17, 512, 512), (17, 1024, 8192), (33, 512, 512), (33, 1024, 8192),
           (16, 8192, 1024), (1, 5120, 27648), (32, 8192, 1024), (32, 1024, 8192), (33, 12000, 2000), (33, 4096, 4096),
           (8, 27648, 5120), (16, 8192, 8192), (17, 27648, 5120), (17, 8192, 8192),
           (49, 512, 512), (49, 2048, 2048), (300, 8192, 1024), (384, 2048, 2048), (1500, 4096, 4096),
           (200, 27648, 5120), (49, 27648, 5120), (1024, 8192, 1024), (1024, 12000, 2000), (700, 12000, 2000),
           (384, 27648, 5120), (3000, 700, 20000), (1500, 8192, 1024), (1500, 12000, 2000), (1024, 27648, 5120),
           (512, 27648, 5120), (4096, 700, 20000), (2048, 8192, 1024), (2048, 12000, 2000), (3000, 27648, 5120)]
BACKWARD = [(1, 512, 512), (1, 2048, 2048), (17, 512, 512), (17, 2048, 2048), (16, 27648, 5120), (32, 27648, 5120),
            (33, 512, 512), (33, 2048, 2048), (80, 700, 20000), (80, 1024, 8192), (8192, 512, 512), (100, 4096, 4096),
            (1024, 1024, 8192), (300, 5120, 27648), (512, 700, 20000), (160, 8192, 8192), (1500, 1024, 8192),
            (1024, 700, 20000), (700, 700, 20000), (100, 5120, 27648), (2048, 1024, 8192), (1500, 700, 20000),
            (700, 5120, 27648)]


@pytest.fixture(scope="module")
def b():
    from dora_fine_tuning_amd import binding

    return binding


def case(b, T, out, in_, dtype, K):
    g = torch.Generator(device=DEV)
    g.manual_seed(T * 7919 + out * 31 + in_)
    W = (torch.randn((out, in_), generator=g, device=DEV) * 0.02).to(DT[dtype])
    return (*b.dora_q4_pack_weight(W), torch.randn((T, K), generator=g, device=DEV).to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("T,out,in_", FORWARD)
def test_forward(b, T, out, in_, odd, dtype):
    if odd:
        T, out, in_ = max(1, T - T // 20), out - 5, in_ - 3
    q, e, x = case(b, T, out, in_, dtype, in_)
    y = b.dora_q4_linear_fwd(x, q, e, out)
    assert_product(y, x, values(b, q, e, out, in_).t())
    assert torch.equal(b.dora_q4_linear_fwd(x, q, e, out), y)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("T,out,in_", BACKWARD)
def test_backward(b, T, out, in_, odd, dtype):
    if odd:
        T, out, in_ = max(1, T - T // 20), out - 3, in_ - 5
    q, e, g = case(b, T, out, in_, dtype, out)
    dx = b.dora_q4_linear_bwd(g, q, e, in_)
    assert_product(dx, g, values(b, q, e, out, in_))
    assert torch.equal(b.dora_q4_linear_bwd(g, q, e, in_), dx)
