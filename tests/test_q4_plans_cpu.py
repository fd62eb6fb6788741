"""Which kernel sizes ask for: the lists that stand for every kernel do so."""
import math
import random

import pytest

from dora_fine_tuning_amd import binding
from q4_plans import BACKWARD, FORWARD, KINDS, NORM, SIZES, kind_of


@pytest.mark.parametrize("product,kind,T,out,in_", SIZES)
def test_sizes_take_their_kernel(product, kind, T, out, in_):
    assert kind_of(T, out, in_, product) == kind


@pytest.mark.parametrize("product", [FORWARD, BACKWARD, NORM])
def test_no_size_takes_another_kernel(product):
    rng = random.Random(product)
    lg = lambda a, b: int(math.exp(rng.uniform(math.log(a), math.log(b))))
    unknown = {}
    for _ in range(40000):
        T, out, in_ = 8 * rng.randint(1, 64) if product == NORM else lg(1, 20000), lg(1, 60000), lg(1, 60000)
        if product == NORM:
            in_ = max(8, in_ // 8 * 8)
        if rng.random() < 0.5:
            out, in_ = max(64, out // 64 * 64), max(64, in_ // 64 * 64)
        kind = kind_of(T, out, in_, product)
        if kind not in KINDS[product]:
            unknown[kind] = (T, out, in_)
    assert not unknown


def test_the_lists_of_the_gpu_tests_take_every_kernel_that_they_name():
    """The tests with random operands run on these; the sharings that they miss, on SIZES."""
    import test_q4_kernels_gpu as K
    import test_q4_norm_gpu as N

    geometry = lambda kind: kind[:-1]
    for product, sizes in ((FORWARD, K.FORWARD), (BACKWARD, K.BACKWARD), (NORM, [(r, o, i) for o, i, r in N.EVERY])):
        taken = {kind_of(*s, product) for s in sizes}
        assert {geometry(k) for k in taken} == {geometry(k) for k in KINDS[product]}, product
        assert taken <= set(KINDS[product])


def test_plan_numbers():
    assert binding.dora_q4_plan(8192, 8192, 8192, FORWARD) == (128, 256, 2048, 0, 1, 512)
    rows, cols, whole, rest, ranges, grid = binding.dora_q4_plan(300, 8192, 8192, BACKWARD)
    assert (whole + rest) == -(-300 // rows) * (8192 // cols) and grid <= 768 and grid % 8 == 0
    for empty in ((0, 8, 8), (8, 0, 8), (8, 8, 0)):
        assert binding.dora_q4_plan(*empty, FORWARD) == (0,) * 6


def test_plan_refusals():
    call = lambda T=8, out=64, in_=64, product=0, plan=1 << 40: binding.LIB.dora_q4_plan(T, out, in_, product, plan)
    for kw, status, text in (({"T": -1}, binding.DORA_INVALID_ARG, "negative"),
                             ({"plan": None}, binding.DORA_INVALID_ARG, "NULL"),
                             ({"product": 3}, binding.DORA_INVALID_ARG, "product"),
                             ({"out": 1 << 22}, binding.DORA_UNSUPPORTED, "beyond"),
                             ({"T": 12, "product": 2}, binding.DORA_UNSUPPORTED, "norm"),
                             ({"T": 0, "product": 2}, binding.DORA_UNSUPPORTED, "norm")):
        assert call(**kw) == status and text in binding.dora_last_error(), kw
