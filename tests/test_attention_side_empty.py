"""Calls of the attention side for no sequences (no GPU)."""
import bit_vq_routed_gb300 as bv
from test_attention_side_args import _attention


def test_no_sequences():
    # T = 0 enqueues nothing, whether the batch has idle sequences or none
    lib = bv.load()
    n = bv.moe_launch_count()
    assert _attention(lib, T=0, B=0, q=None, max_pages=0, page_table=None) == bv.MOE_OK
    assert _attention(lib, T=0, B=-1) == bv.MOE_ERR_INVALID_ARG
    assert _attention(lib, T=1, B=0) == bv.MOE_ERR_INVALID_ARG
    assert bv.moe_launch_count() == n
