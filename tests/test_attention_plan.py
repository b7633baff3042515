"""plan_batch: the host arrays of a step (no GPU needed)."""
import numpy as np
import pytest

import bit_vq_routed_gb300 as bv


def test_arrays():
    pos, slots, cu, pp, table, lens = bv.plan_batch(8, [5, 2], 13, [[7, 3], [4], [9, 1, 0]], [6, 0, 15], [4, 2, 0])
    assert pos.tolist() == [19, 20, 21, 22, 13, 14] and pos.dtype == np.int32
    assert slots.tolist() == [7 * 8 + 6, 7 * 8 + 7, 3 * 8, 3 * 8 + 1, 4 * 8, 4 * 8 + 1] and slots.dtype == np.int64
    assert cu.tolist() == [0, 4, 6, 6] and pp.tolist() == [5, 2]
    assert table.tolist() == [[7, 3, 0], [4, 0, 0], [9, 1, 0]]
    assert lens.tolist() == [10, 2, 15] and lens.dtype == np.int32


def test_slots_past_32_bits():
    _, slots, *_ = bv.plan_batch(1024, [], 0, [[1 << 22]], [1023], [1])
    assert slots.tolist() == [(1 << 32) + 1023]


def test_empty_batch():
    pos, slots, cu, pp, table, lens = bv.plan_batch(16, [], 0, [[], [3]], [0, 5], [0, 0])
    assert pos.size == slots.size == pp.size == 0 and cu.tolist() == [0, 0, 0]
    assert table.shape == (2, 1) and lens.tolist() == [0, 5]


def test_too_few_pages():
    with pytest.raises(ValueError, match="sequence 1"):
        bv.plan_batch(8, [], 0, [[0], [1]], [0, 7], [1, 2])
    with pytest.raises(ValueError, match="prefix"):
        bv.plan_batch(8, [3], 9, [[0]], [0], [1])
    with pytest.raises(ValueError, match="one entry"):
        bv.plan_batch(8, [], 0, [[0]], [0], [1, 1])
