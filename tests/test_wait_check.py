"""A device-side wait that gave up, as the caller learns of it (the word is set
here by hand: no wait is made to run out)."""
import pytest
import torch

import bit_vq_routed_gb300 as bv


def _set(ws, code):
    ws[8:12].view(torch.int32).fill_(code)


def test_raises_once_for_a_noted_wait():
    ws = torch.zeros(256, dtype=torch.uint8)
    bv.moe_check_waits(ws)
    for code in (1, 2):
        _set(ws, code)
        with pytest.raises(bv.MoeError, match=f"code {code}") as e:
            bv.moe_check_waits(ws)
        assert e.value.status == bv.MOE_ERR_TIMEOUT
        bv.moe_check_waits(ws)
    assert not bool(ws.any())


def test_layer_looks_at_both_workspaces():
    layer = bv.AttentionLayer.__new__(bv.AttentionLayer)
    layer.ws, layer.attn_ws = (torch.zeros(256, dtype=torch.uint8) for _ in range(2))
    layer.check()
    for ws, what in ((layer.ws, "projections"), (layer.attn_ws, "attention")):
        _set(ws, 1)
        with pytest.raises(bv.MoeError, match=what):
            layer.check()
        layer.check()


@pytest.mark.gpu
def test_after_a_step():
    bf = dict(dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.zeros(8, 16, 2, 64, **bf) for _ in range(2))
    layer = bv.AttentionLayer(8, 2, 64, torch.randn(12 * 64, 256, **bf), None, torch.randn(256, 512, **bf), kc, vc, 4,
                              bv.rotation_table(64, 64))
    x = torch.randn(4, 256, **bf)
    batch = bv.upload_batch(16, [], 0, [[0], [1]], [0, 0], [3, 1])
    want = layer.forward(x, batch).clone()
    layer.check()
    for ws in (layer.ws, layer.attn_ws):
        _set(ws, 2)  # (as a call would leave it)
        layer.forward(x, batch)
        with pytest.raises(bv.MoeError):
            layer.check()
    assert torch.equal(layer.forward(x, batch), want)  # the workspaces serve on
    layer.check()
