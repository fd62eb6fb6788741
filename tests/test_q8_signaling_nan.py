"""Packing of signaling NaN: such a value is stored as NaN and does not count for
its block's exponent, wherever it stands beside the block's largest value.  The
bytes are equal to the oracle's, so there is no tolerance."""
import numpy as np
import pytest
import torch

from oracle import dora_oracle as O
from oracle import q8_oracle as Q

F = pytest.importorskip("dora_fine_tuning_amd.torch_ops")
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
SIGNALING = {"bf16": 0x7F81, "fp16": 0x7C01}  # all exponent bits, the fraction's top bit clear


def rows_with_signaling_nan(dtype):
    """A row for every pair of places (NaN, largest value) among eight neighbours
    (what one lane holds), both signs, the NaN once alone in its block too."""
    rng = np.random.default_rng(12)
    rows = []
    for nan in range(8):
        for big in range(8):
            for sign in (0, 0x8000):
                v = torch.from_numpy(rng.standard_normal(300).astype(np.float32)).to(DT[dtype])
                lane = 8 * int(rng.integers(0, 16))
                v[lane + big] = 1000.0
                bits = v.view(torch.int16).numpy()
                word = np.array(SIGNALING[dtype] | sign, np.uint16).view(np.int16)
                bits[lane + nan] = word
                bits[128 + lane + nan] = word  # the next block: no value stands out
                bits[256 + nan:300] = 0
                bits[256 + nan] = word  # alone among zeros
                rows.append(v)
    return torch.stack(rows)


def check(dtype, device):
    x = rows_with_signaling_nan(dtype)
    for pack, oracle in ((F.q8_pack, Q.pack_rows), (F.q8_pack_weight, Q.pack_weight)):
        q, e = pack(x.to(device))
        q = q.view(torch.uint8).cpu().numpy()
        rq, re_ = oracle(O.as_f64(x))
        assert np.array_equal(e.cpu().numpy(), re_)
        nan = np.isnan(Q.E4M3[rq])
        assert np.array_equal(np.isnan(Q.E4M3[q]), nan) and np.array_equal(q[~nan], rq[~nan])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_signaling_nan_eager(dtype):
    check(dtype, "cpu")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_signaling_nan(dtype):
    check(dtype, "cuda:0")
