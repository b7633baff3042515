"""The attention side end to end: a prompt in chunks and then single tokens,
against the same layer in 64 bits (with the roundings between its steps), and
with the routed experts behind it."""
import math

import numpy as np
import pytest

import moe_synth as ms
from gpu_common import assert_close, device_layer, torch_cuda

pytestmark = pytest.mark.gpu

H, QH, KVH, D, PAGE = 256, 8, 2, 64, 16


def _layer(torch, dtype, T_max, rot=D, inter=False, seed=0):
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    g = ac.gen(seed)
    w_qkv = ac.normal(g, (QH + 2 * KVH) * D, H, dtype=dtype, std=H ** -0.5)
    b_qkv = ac.normal(g, (QH + 2 * KVH) * D, dtype=dtype, std=0.1)
    w_out = ac.normal(g, H, QH * D, dtype=dtype, std=(QH * D) ** -0.5)
    kc = torch.full((64, PAGE, KVH, D), float("nan"), dtype=dtype, device="cuda")
    vc = kc.clone()
    return bv.AttentionLayer(QH, KVH, D, w_qkv, b_qkv, w_out, kc, vc, T_max, bv.rotation_table(2048, rot), inter)


def _turn(torch, x, pos, rot, inter):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = pos.double()[:, None, None] * f
    x = x.double().clone()
    ia = torch.arange(0, rot, 2) if inter else torch.arange(rot // 2)
    ib = ia + 1 if inter else ia + rot // 2
    p, q = x[..., ia], x[..., ib]
    x[..., ia], x[..., ib] = p * a.cos() - q * a.sin(), q * a.cos() + p * a.sin()
    return x


def _dense(torch, layer, x, residual, start, past, rot, inter):
    """One sequence without a cache: x [n, H] behind `past` (turned keys, values
    in the element type); returns (output, new past)."""
    dt = layer.w_qkv.dtype
    qkv = (x.double() @ layer.w_qkv.double().t() + layer.b_qkv.double()).to(dt).view(-1, QH + 2 * KVH, D)
    pos = torch.arange(start, start + x.shape[0], device="cuda")
    q = _turn(torch, qkv[:, :QH], pos, rot, inter).to(dt)
    k = torch.cat((past[0], _turn(torch, qkv[:, QH:QH + KVH], pos, rot, inter).to(dt)))
    v = torch.cat((past[1], qkv[:, QH + KVH:]))
    n, m = x.shape[0], k.shape[0]
    s = torch.einsum("qhd,khd->hqk", q.double(), k.double().repeat_interleave(QH // KVH, 1)) / math.sqrt(D)
    s = s.masked_fill(torch.arange(m, device="cuda") > (m - n + torch.arange(n, device="cuda"))[:, None], -math.inf)
    a = torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), v.double().repeat_interleave(QH // KVH, 1)).to(dt)
    y = a.reshape(n, -1).double() @ layer.w_out.double().t()
    return y + residual.double(), (k, v)


@pytest.mark.parametrize("dtype,rot,inter", [("bfloat16", 64, False), ("float16", 32, True)])
def test_prefix_then_prompts_then_tokens(dtype, rot, inter):
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    dt = getattr(torch, dtype)
    layer = _layer(torch, dt, 200, rot, inter)
    g = ac.gen(3)
    # Tolerance: an output is a sum of QH * D = 512 products of attention values of about 1 and weights
    # of about 512^-1/2, so of size 1; each attention value carries up to 2 u of its own size (its rounding,
    # the probabilities') where both sides round q, k and v alike, except where the two sides round apart (one
    # u, in few places): 4 u in all, in quadrature over the sum well below 8 u of the result's own scale.
    tol = 8 * ac.U[dt]

    def check(got, want, what):
        err = (got.double() - want).abs().max() / want.abs().mean()
        assert float(err) <= tol, (what, float(err), tol)

    none = torch.empty(0, KVH, D, dtype=dt, device="cuda")
    # the shared prefix of 37 tokens, as the only sequence of a call
    prefix_pages = [11, 3, 40]
    x = ac.normal(g, 37, H, dtype=dt)
    r = ac.normal(g, 37, H, dtype=dt)
    b = bv.upload_batch(PAGE, [], 0, [prefix_pages], [0], [37])
    got = layer.forward(x, b, r)
    want, shared = _dense(torch, layer, x, r, 0, (none, none), rot, inter)
    check(got, want, "prefix")
    # prompts of three sequences behind it, in two chunks, then single tokens
    pages = [[1, 2, 5, 7, 8], [20, 21], [30, 33, 31, 32]]
    lens = [0, 0, 0]
    past = [shared] * 3
    for new in ([40, 0, 20], [33, 5, 30], [1, 1, 1], [1, 1, 1]):
        T = sum(new)
        x, r = ac.normal(g, T, H, dtype=dt), ac.normal(g, T, H, dtype=dt)
        got = layer.forward(x, bv.upload_batch(PAGE, prefix_pages, 37, pages, lens, new), r).clone()
        t = 0
        for s, n in enumerate(new):
            if n:
                want, past[s] = _dense(torch, layer, x[t:t + n], r[t:t + n], 37 + lens[s], past[s], rot, inter)
                check(got[t:t + n], want, f"sequence {s} of {new}")
            lens[s] += n
            t += n
    assert int(layer.ws[8:12].view(torch.int32).item()) == 0
    assert int(layer.attn_ws[8:12].view(torch.int32).item()) == 0


def test_decoder_layer_and_graph():
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    import oracle
    lay = ms.Layer(ms.spec_tiny(0))
    dev, _keep = device_layer(lay, 4)
    layer = bv.DecoderLayer(_layer(torch, torch.bfloat16, 40), dev)
    g = ac.gen(9)
    prefix_pages = [11, 3, 40]
    layer.attention.forward(ac.normal(g, 37, H), bv.upload_batch(PAGE, [], 0, [prefix_pages], [0], [37]))
    pages = [[1], [2], [5], [7]]
    x, r = ac.normal(g, 4, H), ac.normal(g, 4, H, std=0.5)
    batch = bv.upload_batch(PAGE, prefix_pages, 37, pages, [0] * 4, [1] * 4)
    h, y = layer.forward(x, batch, r)
    torch.cuda.synchronize()
    bits = h.view(torch.uint16 if hasattr(torch, "uint16") else torch.int16).cpu().numpy().view(np.uint16)
    ref = oracle.default.moe_layer(lay, bits)  # the experts of the very activations that reached them
    assert np.array_equal(dev.ids[:4].cpu().numpy(), ref["ids"])
    assert_close(y.cpu().numpy(), ref["out"])
    # the same step as a graph, then the next token through it (lengths and slots read anew)
    h0, y0 = h.clone(), y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, batch, r)
    graph.replay()
    assert torch.equal(layer.attention.out[:4], h0) and torch.equal(dev.out[:4], y0)
    nxt = bv.upload_batch(PAGE, prefix_pages, 37, pages, [1] * 4, [1] * 4)
    for name in ("positions", "slots", "page_table", "seq_lens"):
        getattr(batch, name).copy_(getattr(nxt, name))
    graph.replay()
    h1 = layer.attention.out[:4].clone()
    h2 = layer.attention.forward(x, nxt, r)  # (writes the same keys and values again)
    assert torch.equal(h1, h2) and not torch.equal(h1, h0)


def test_refuses_shapes():
    torch = torch_cuda()
    import bit_vq_routed_gb300 as bv
    layer = _layer(torch, torch.bfloat16, 4)
    with pytest.raises(ValueError, match="T_max"):
        layer.forward(torch.zeros(5, H, dtype=torch.bfloat16, device="cuda"), None)
    with pytest.raises(ValueError, match="do not fit"):
        bv.AttentionLayer(QH, KVH, D, layer.w_qkv, None, layer.w_out[:, 8:], layer.k_cache, layer.v_cache, 4)
