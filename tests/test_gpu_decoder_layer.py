"""DecoderLayer as a pre-norm layer: RMS norms ahead of the attention side and of
the experts, eagerly and as a captured step, against its parts called apart."""
import numpy as np
import pytest

import moe_synth as ms
from gpu_common import assert_close, device_layer, torch_cuda

pytestmark = pytest.mark.gpu

QH, KVH, D, PAGE = 8, 2, 64, 16


def _setup(torch, T_max):
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    lay = ms.Layer(ms.spec_tiny(0))
    dev, keep = device_layer(lay, T_max)
    H, g = dev.H, ac.gen(1)
    w_qkv = ac.normal(g, (QH + 2 * KVH) * D, H, std=H ** -0.5)
    w_out = ac.normal(g, H, QH * D, std=(QH * D) ** -0.5)
    kc, vc = (torch.zeros(16, PAGE, KVH, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    att = bv.AttentionLayer(QH, KVH, D, w_qkv, None, w_out, kc, vc, T_max, bv.rotation_table(512, D))
    gains = [ac.normal(g, H).float() * 0.1 + 1 for _ in range(2)]

    def norm(gain):
        def f(h):
            v = h.float()
            return (v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * gain).to(torch.bfloat16)
        return f

    return lay, dev, keep, att, norm(gains[0]), norm(gains[1])


@pytest.mark.parametrize("T", [1, 4, 20])
def test_pre_norm_layer(T):
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    import oracle
    lay, dev, keep, att, norm1, norm2 = _setup(torch, 20)
    block = bv.DecoderLayer(att, dev, norm=norm2)
    x = ac.normal(ac.gen(2), T, dev.H)
    batch = bv.upload_batch(PAGE, [], 0, [[b] for b in range(T)] if T <= 4 else [[5, 6]], [0] * (T if T <= 4 else 1),
                            [1] * T if T <= 4 else [T])
    h, y = (t.clone() for t in block.forward(norm1(x), batch, residual=x))
    # the parts apart, with a wait for the device between them
    h2 = att.forward(norm1(x), batch, residual=x)
    torch.cuda.synchronize()
    z = norm2(h2)
    torch.cuda.synchronize()
    y2 = dev.forward(z)
    assert torch.equal(h, h2) and torch.equal(y, y2)
    bits = z.view(torch.int16).cpu().numpy().view(np.uint16)
    ref = oracle.default.moe_layer(lay, bits)
    assert np.array_equal(dev.ids[:T].cpu().numpy(), ref["ids"])
    assert_close(y.cpu().numpy(), ref["out"])
    # on another stream, as an object and as a handle
    other = torch.cuda.Stream()
    z1 = norm1(x)
    for stream in (other, other.cuda_stream):
        torch.cuda.synchronize()
        h2, y2 = block.forward(z1, batch, residual=x, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(h, h2) and torch.equal(y, y2)
    # as a captured step whose tokens change from replay to replay
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hg, yg = block.forward(norm1(static), batch, residual=static)
    for i in range(5):
        new = ac.normal(ac.gen(10 + i), T, dev.H)
        static.copy_(new)
        graph.replay()
        hr, yr = hg.clone(), yg.clone()
        h2 = att.forward(norm1(new), batch, residual=new)
        torch.cuda.synchronize()
        z = norm2(h2)
        torch.cuda.synchronize()
        assert torch.equal(hr, h2) and torch.equal(yr, dev.forward(z)), i
