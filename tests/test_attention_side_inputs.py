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


@pytest.mark.parametrize("kw", [dict(lens=[3, -1]), dict(new=[-2, 1]), dict(prefix_len=-1), dict(page_size=0)])
def test_plan_refuses_negative_numbers(kw):
    # (they would give positions below zero, and token ranges that go backwards)
    a = dict(page_size=8, prefix_pages=[5], prefix_len=3, pages=[[0], [1]], lens=[3, 1], new=[1, 1])
    bv.plan_batch(**a)
    a.update(kw)
    with pytest.raises(ValueError, match="negative"):
        bv.plan_batch(**a)
