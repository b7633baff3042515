"""Sizes next to the largest int are refused, where rounding them up to whole tiles
would leave its range (no GPU needed)."""
import ctypes
import struct

import pytest

import bit_vq_routed_gb300 as bv

P = ctypes.c_void_p(4096)
MAX = 2 ** 31 - 1


@pytest.mark.parametrize("T,N", [(MAX, 1), (MAX - 14, 1), (MAX - 100, 1), (1, MAX), (1, MAX - 100), (1, MAX - 126), (20, MAX - 5)])
def test_products(T, N):
    lib = bv.load()
    n = bv.moe_launch_count()
    assert lib.moe_linear(P, 16, P, 16, None, None, 0, P, N, T, N, 16, 0, 0, P, 256, None) == bv.MOE_ERR_UNSUPPORTED
    assert b"moe_linear" in lib.moe_last_error()
    assert lib.moe_linear_8bit(P, 16, P, P, 16, P, None, None, 0, P, N, T, N, 16, 0, 0, P, 256, None) == bv.MOE_ERR_UNSUPPORTED
    assert b"moe_linear_8bit" in lib.moe_last_error()
    assert bv.moe_launch_count() == n


@pytest.mark.parametrize("T", [MAX, MAX - 1, MAX - 2])
def test_choice(T):
    lib = bv.load()
    n = bv.moe_launch_count()
    how = struct.pack("@iifP3i4x", 1, 1, 1.0, 0, 1, 1, 1)
    assert lib.moe_route_scored(P, T, 1, 1, how, P, P, None) == bv.MOE_ERR_UNSUPPORTED
    assert bv.moe_launch_count() == n
