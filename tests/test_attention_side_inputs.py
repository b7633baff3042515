"""What AttentionLayer's helpers refuse (no GPU)."""
import pytest

import bit_vq_routed_gb300 as bv


@pytest.mark.parametrize("rot", [1, 5, 63, -2])
def test_rotation_table_refuses_odd_sizes(rot):
    # (a table of rot + 1 columns would turn one element more, by other angles)
    with pytest.raises(ValueError, match="rot_dim"):
        bv.rotation_table(16, rot, device="cpu")


def test_rotation_table_sizes():
    for rot in (0, 2, 64):
        assert tuple(bv.rotation_table(16, rot, device="cpu").shape) == (16, rot)
