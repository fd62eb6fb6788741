"""Every kernel of the 4-bit products and every way in which it shares out its work, at
the sizes that test_q4_plans_cpu holds to it: the products bit for bit (q4_exact), the
norm against 64 bits (tolerance in test_q4_norm_gpu)."""
import pytest
import torch

from q4_exact import assert_exact, rows, weight
from q4_plans import BACKWARD, FORWARD, NORM, SIZES, kind_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def b():
    from dora_fine_tuning_amd import binding

    return binding


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("product,kind,T,out,in_", [s for s in SIZES if s[0] in (FORWARD, BACKWARD)])
def test_products(b, product, kind, T, out, in_, dtype):
    assert kind_of(T, out, in_, product) == kind
    W = weight(out, in_, DEV)
    q, e = b.dora_q4_pack_weight(W.to(DT[dtype]))
    x = rows(T, in_ if product == FORWARD else out, DEV)
    call, n = (b.dora_q4_linear_fwd, out) if product == FORWARD else (b.dora_q4_linear_bwd, in_)
    assert_exact(call(x.to(DT[dtype]), q, e, n), x, W.t() if product == FORWARD else W, (T, out, in_))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("product,kind,r,out,in_", [s for s in SIZES if s[0] == NORM])
def test_norm(b, product, kind, r, out, in_, dtype):
    assert kind_of(r, out, in_, NORM) == kind
    g = torch.Generator(device=DEV)
    g.manual_seed(out + r)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV).to(DT[dtype])
    q, e = b.dora_q4_pack_weight(rand(out, in_) * 0.02)
    W = b.dora_q4_unpack_weight(q, e, out, in_, DT[dtype])
    A, B, c = rand(r, in_) * 0.02, rand(out, r) * 0.02, b.dora_row_sqnorm(W)
    got = b.dora_q4_norm_cached(q, e, A, B, c, 2.0).double()
    V = B.double() @ A.double()
    n = (c.double() + (4.0 * W.double() * V + 4.0 * V * V).sum(dim=1)).sqrt()
    assert bool(((got - n).abs() <= 1e-5 * n).all()), (got / n - 1).abs().max()
