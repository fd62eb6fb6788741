"""The token slices of the 8-bit backward keep every operand's slice below 2 GiB,
the packed rows' too: its offsets are 32-bit.  Read from the workspace, which
holds one fp32 slice of the sums a token slice."""
import pytest

from dora_fine_tuning_amd import binding

LIB = binding.LIB


@pytest.mark.parametrize("cols", [1, 8, 63, 64, 65, 200, 4096])
@pytest.mark.parametrize("r", [8, 64])
@pytest.mark.parametrize("T", [(1 << 31) - 1, (1 << 30) + 5, 1 << 20])
def test_slices_stay_below_2_gib(T, r, cols):
    packed, rows16 = -(-cols // 128) * 128, -(-cols // 8) * 16
    for query, widest in ((LIB.dora_q8_lora_compose_bwd_workspace_bytes, max(packed, rows16, 2 * r)),
                          (LIB.dora_q8_grad_a_workspace_bytes, max(packed, 2 * r))):
        need = query(T, cols, r)
        if query is LIB.dora_q8_lora_compose_bwd_workspace_bytes and cols % 8:
            need -= T * rows16  # dy's padded copy
        slices = (need + 4096) // (cols * r * 4)  # an upper bound: the partials take room too
        exact = -(-T // (((1 << 31) - 1) // widest))
        assert slices >= exact, (slices, exact)
