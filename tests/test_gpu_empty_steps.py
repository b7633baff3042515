"""Steps without tokens, or without sequences, through AttentionLayer and DecoderLayer: nothing is
launched by the attention side and nothing is written."""
import pytest

import moe_synth as ms
from gpu_common import device_layer, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [0, 1, 3])
def test_no_tokens(B):
    torch = torch_cuda()
    import bit_vq_routed_gb300 as bv
    dev, _keep = device_layer(ms.Layer(ms.spec_tiny(0)), 4)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.full((8, 16, 2, 64), 7.0, **bf) for _ in range(2))
    att = bv.AttentionLayer(8, 2, 64, torch.zeros(12 * 64, dev.H, **bf), None, torch.zeros(dev.H, 512, **bf), kc, vc, 4,
                            bv.rotation_table(64, 64))
    att.out.fill_(7.0)
    x = torch.empty(0, dev.H, **bf)
    batch = bv.upload_batch(16, [0], 9, [[b + 1] for b in range(B)], [b for b in range(B)], [0] * B)
    n = bv.moe_launch_count()
    assert tuple(att.forward(x, batch).shape) == (0, dev.H)
    assert tuple(att.forward(x, batch, residual=x).shape) == (0, dev.H)
    assert bv.moe_launch_count() == n
    h, y = bv.DecoderLayer(att, dev).forward(x, batch, residual=x)
    assert tuple(h.shape) == (0, dev.H) and tuple(y.shape) == (0, dev.H)
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in (kc, vc, att.out))
