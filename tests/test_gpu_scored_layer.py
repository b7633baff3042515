"""The norm, the 8-bit projections and the choice by score in the layers that use
them: the whole routing in one call, a MoELayer that chooses by score, and two
decoder layers one behind the other, each stage against 64 bits."""
import pytest

torch = pytest.importorskip("torch")
import attn_common as ac  # noqa: E402
import moe_synth as ms  # noqa: E402
import rows_common as rc  # noqa: E402
from gpu_common import experts_fn, torch_cuda  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _i(*s):
    return torch.full(s, -7, dtype=I32, device="cuda")


def _f(*s):
    return torch.full(s, -7.0, device="cuda")


@pytest.mark.parametrize("E,k,groups,top_groups", [(8, 2, 4, 2), (256, 8, 8, 4), (60, 5, 1, 1), (1024, 32, 16, 4)])
@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 65, 1100])
@pytest.mark.parametrize("fresh", [False, True])
def test_the_whole_routing_is_its_three_steps(T, E, k, groups, top_groups, fresh):
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    g = ac.gen(T + E)
    H = 512
    x, w = ac.normal(g, T, H), ac.normal(g, E, H, std=0.05)
    rb, bias = ac.normal(g, E, dtype=F32, std=0.1), ac.normal(g, E, dtype=F32, std=0.05)
    how = dict(scoring=bv.MOE_SCORE_SIGMOID, bias=bias, groups=groups, top_groups=top_groups, group_top=2 if groups > 1 else 1,
               renormalize=1, scale=2.5)

    def outs():
        return _f(T, E), _i(T, k), _f(T, k), _i(E + 1), _i(T * k), _i(T * k)

    a, b = outs(), outs()
    ws = torch.empty(max(16, bv.moe_permute_workspace_size(T, k, E)), dtype=torch.uint8, device="cuda")
    bv.moe_route_tokens_scored(x, w, rb, k, *a, ws=ws, fresh=fresh, **how)
    bv.moe_router_logits(x, w, rb, b[0])
    bv.moe_route_scored(b[0], k, b[1], b[2], **how)
    bv.moe_permute(b[1], E, *b[3:])
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_no_tokens():
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    off = _i(17)
    bv.moe_route_tokens_scored(torch.zeros(0, 256, dtype=BF, device="cuda"), ac.normal(ac.gen(0), 16, 256), None, 2, _f(0, 16),
                               _i(0, 2), _f(0, 2), off, _i(0), _i(0), scoring=1)
    assert off.tolist() == [0] * 17


def _moe(T_max, layer=0, **scoring):
    import bit_vq_routed_gb300 as bv
    lay = ms.Layer(ms.spec_tiny(layer))
    s = lay.spec
    return bv.upload_layer(s.H, s.I, s.E, s.k, T_max, lay.codebook, lay.w_router, lay.bias, experts_fn(lay), s.renormalize,
                           scoring=bv.Scoring(**scoring))


def _routed(moe, T, bias, groups, top_groups, group_top, scale):
    """The last forward's experts, weights and combine, from its own logits."""
    ids, w = rc.scored64(moe.logits[:T], moe.k, True, bias, groups, top_groups, group_top, moe.renormalize, scale)
    assert torch.equal(moe.ids[:T].cpu(), ids)
    ac.within(moe.weights[:T].cpu(), w, w.abs() * 64 * 2.0 ** -23 + 2.0 ** -120, "router weights")
    y = moe.ypair[moe.pair_to_sorted[:T * moe.k].long()].view(T, moe.k, -1).double()
    terms = moe.weights[:T].double()[..., None] * y
    ac.within(moe.out[:T], terms.sum(1), 4 * moe.k * 2.0 ** -23 * terms.abs().sum(1), "combine")


@pytest.mark.parametrize("T", [1, 4, 40])
def test_layer_that_chooses_by_score(T):
    torch_cuda()
    bias = ac.normal(ac.gen(3), 8, dtype=F32, std=0.2)
    dev, keep = _moe(40, bias=bias, groups=4, top_groups=2, group_top=2, scale=1.5)
    x = ac.normal(ac.gen(T), T, dev.H)
    out = dev.forward(x).clone()
    _routed(dev, T, bias, 4, 2, 2, 1.5)
    # a bias that keeps all but two groups' experts out, put in place
    bias.fill_(-float("inf"))
    bias[2:6] = 0
    dev.forward(x)
    assert set(dev.ids[:T].flatten().tolist()) <= {2, 3, 4, 5}
    _routed(dev, T, bias, 4, 2, 2, 1.5)
    bias.copy_(ac.normal(ac.gen(3), 8, dtype=F32, std=0.2))
    # captured, the tokens and the bias change from replay to replay
    import bit_vq_routed_gb300 as bv
    step = bv.GraphedForward(dev, T)
    step.x.copy_(x)
    assert torch.equal(step.replay(), out)
    bias.neg_()
    step.x.copy_(ac.normal(ac.gen(T + 1), T, dev.H))
    step.replay()
    _routed(dev, T, bias, 4, 2, 2, 1.5)
    # the three separate calls give the same routing
    ids, w = dev.ids[:T].clone(), dev.weights[:T].clone()
    dev.route_stepwise(step.x)
    assert torch.equal(ids, dev.ids[:T]) and torch.equal(w, dev.weights[:T])


# ------------------------------------------------------------------ decoder layers

QH, KVH, D, PAGE = 8, 2, 64, 16


def _decoder(n, T_max, eight):
    import bit_vq_routed_gb300 as bv
    bias = ac.normal(ac.gen(20 + n), 8, dtype=F32, std=0.1)
    moe, keep = _moe(T_max, n, bias=bias, groups=2, top_groups=1, group_top=2, scale=2.0)
    H, g = moe.H, ac.gen(30 + n)
    w_qkv, w_out = ac.normal(g, (QH + 2 * KVH) * D, H, std=H ** -0.5), ac.normal(g, H, QH * D, std=(QH * D) ** -0.5)
    kc, vc = (torch.zeros(16, PAGE, KVH, D, dtype=BF, device="cuda") for _ in range(2))
    if eight:
        w_qkv, w_out = bv.quantize_rows(w_qkv), bv.quantize_rows(w_out)
    gains = [(1 + ac.normal(g, H, dtype=F32, std=0.1)).to(BF) for _ in range(2)]
    att = bv.AttentionLayer(QH, KVH, D, w_qkv, ac.normal(g, (QH + 2 * KVH) * D), w_out, kc, vc, T_max)
    return bv.DecoderLayer(att, moe, norm=bv.RMSNorm(gains[1], 1e-6, T_max),
                           norm_in=bv.RMSNorm(gains[0], 1e-5, T_max, eight=eight)), bias, keep


def _check_layer(block, bias, batch, h_in, y_in, h, y, eight):
    """Every stage of a step from what it read."""
    att, T = block.attention, h.shape[0]
    stream = h_in if y_in is None else (y_in + h_in.float()).to(BF)
    n = block.norm_in
    if y_in is not None:
        assert torch.equal(n.h[:T], stream)
    z64, rel = rc.rms64(stream, n.weight, n.eps)
    if eight:
        rc.check_rows8(n.y.q[:T], n.y.scales[:T], z64, rel, "norm ahead of the attention")
        want, tol = rc.linear8_64(n.y.q[:T], n.y.scales[:T], att.w_qkv.q, att.w_qkv.scales, att.b_qkv, 0, None, BF)
    else:
        ac.within(n.y[:T], z64, z64.abs() * (rel + 2.0 ** -8 * 1.01) + ac.TINY[BF], "norm ahead of the attention")
        want, tol = ac.linear64(n.y[:T], att.w_qkv, att.b_qkv, 0, None)
    qkv = att.qkv[:T]
    ac.within(qkv.reshape(T, -1), want, tol, "q, k, v")
    q, k, v = qkv.split((QH, KVH, KVH), 1)
    assert torch.equal(att.k_cache.view(-1, KVH, D)[batch.slots], k) and torch.equal(att.v_cache.view(-1, KVH, D)[batch.slots], v)
    want, lse, tol, tlse = ac.attention64(q, att.k_cache, att.v_cache, batch.cu_q, batch.prefix_pages, batch.prefix_len,
                                          batch.page_table, batch.seq_lens, att.scale)
    ac.within(att.attn[:T], want, tol, "attention")
    a = att.attn[:T].reshape(T, -1)
    if eight:
        a8, mag = rc.rows8_64(a)
        assert torch.equal(att.attn8.q[:T].double(), rc.eighths(a8))
        want, tol = rc.linear8_64(att.attn8.q[:T], att.attn8.scales[:T], att.w_out.q, att.w_out.scales, None, 0, stream, BF)
    else:
        want, tol = ac.linear64(a, att.w_out, None, 0, stream)
    ac.within(h, want, tol, "stream behind the attention")
    z64, rel = rc.rms64(h, block.norm.weight, block.norm.eps)
    ac.within(block.norm.y[:T], z64, z64.abs() * (rel + 2.0 ** -8 * 1.01) + ac.TINY[BF], "norm ahead of the experts")
    _routed(block.moe, T, bias, 2, 1, 2, 2.0)
    assert torch.equal(y, block.moe.out[:T])


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("T", [1, 4, 20])
def test_two_decoder_layers(T, eight):
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    one, two = (_decoder(n, 20, eight) for n in (0, 1))
    x = ac.normal(ac.gen(T), T, one[0].moe.H)
    seqs = [1] * T if T <= 4 else [12, 0, 8]
    batch = bv.upload_batch(PAGE, [], 0, [[b] for b in range(len(seqs))], [0] * len(seqs), seqs)
    h1, y1 = one[0].step(x, None, batch)
    _check_layer(one[0], one[1], batch, x, None, h1, y1, eight)
    h1, y1 = h1.clone(), y1.clone()
    h2, y2 = two[0].step(h1, y1, batch)
    _check_layer(two[0], two[1], batch, h1, y1, h2, y2, eight)
    want = h2.clone(), y2.clone()
    # both layers as one captured step
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hg, yg = two[0].step(*one[0].step(static, None, batch), batch)
    graph.replay()
    assert torch.equal(hg, want[0]) and torch.equal(yg, want[1])
    # and on another stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    hs, ys = two[0].step(*one[0].step(x, None, batch, stream=side), batch, stream=side)
    side.synchronize()
    assert torch.equal(hs, want[0]) and torch.equal(ys, want[1])
    for b in (one[0], two[0]):
        b.attention.check()


def test_steps_without_tokens_and_refusals():
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    block, bias, keep = _decoder(0, 4, True)
    H = block.moe.H
    none = bv.upload_batch(PAGE, [], 0, [], [], [])
    h, y = block.step(torch.zeros(0, H, dtype=BF, device="cuda"), None, none)
    assert h.shape == (0, H) and y.shape == (0, H)
    five = bv.upload_batch(PAGE, [], 0, [[0]], [0], [5])
    n = bv.moe_launch_count()
    with pytest.raises(ValueError, match="T=5"):
        block.step(torch.zeros(5, H, dtype=BF, device="cuda"), None, five)
    with pytest.raises(ValueError, match="T=5"):
        block.norm_in(torch.zeros(5, H, dtype=BF, device="cuda"))
    with pytest.raises(ValueError, match="norm_in"):
        bv.DecoderLayer(block.attention, block.moe).step(torch.zeros(1, H, dtype=BF, device="cuda"), None, none)
    with pytest.raises(ValueError, match="norm_in"):
        bv.DecoderLayer(block.attention, block.moe, norm_in=bv.RMSNorm(torch.ones(H, dtype=torch.float16, device="cuda"), 0.1, 4))
    assert bv.moe_launch_count() == n
    sixteen, _, keep2 = _decoder(0, 4, False)
    with pytest.raises(ValueError, match="8-bit weights"):
        sixteen.attention.forward(bv.quantize_rows(torch.ones(1, H, dtype=BF, device="cuda")),
                                  bv.upload_batch(PAGE, [], 0, [[0]], [0], [1]))


def test_many_tiles_of_a_product():
    """More tiles than the SM pairs take in two rounds: results leave 16 bytes at a
    time, the last tile's and those of odd strides one by one."""
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    T, K = 2900, 256
    for N, pad in ((6152, 0), (6144, 3), (6200, 8)):
        g = ac.gen(N)
        x, w = ac.normal(g, T, K), ac.normal(g, N, K, std=K ** -0.5)
        res = rc.wide(ac.normal(g, T, N), pad)
        bias = ac.normal(g, N)
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        for r in (None, res):
            y = torch.full((T, N + pad + 8 * (pad > 0)), 9.0, dtype=BF, device="cuda")
            bv.moe_linear(x, w, y[:, :N], bias=bias, residual=r, ws=ws)
            want, tol = ac.linear64(x, w, bias, 0, r)
            ac.within(y[:, :N], want, tol, f"16 bits N={N}")
            assert bool((y[:, N:] == 9).all())
            x8, w8 = bv.quantize_rows(x), bv.quantize_rows(w)
            bv.moe_linear_8bit(x8.q, x8.scales, w8.q, w8.scales, y[:, :N], bias=bias, residual=r, ws=ws)
            want, tol = rc.linear8_64(x8.q, x8.scales, w8.q, w8.scales, bias, 0, r, BF)
            ac.within(y[:, :N], want, tol, f"8 bits N={N}")
            assert bool((y[:, N:] == 9).all())
        bv.moe_check_waits(ws)


def test_fetching_tandem_and_gated_forwards_choose_by_score():
    """The layer's other forms route as its plain forward does."""
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    from gpu_common import assert_close
    T, lay = 6, ms.Layer(ms.LayerSpec(H=512, I=256, E=8, k=2, seed=7))
    s, f = lay.spec, experts_fn(lay)
    how = bv.Scoring(bias=ac.normal(ac.gen(1), s.E, dtype=F32, std=0.2), groups=4, top_groups=2, group_top=2, scale=1.5)
    whole, keep = bv.upload_layer(s.H, s.I, s.E, s.k, T, lay.codebook, lay.w_router, lay.bias, f, scoring=how)
    x = ac.normal(ac.gen(2), T, s.H)
    want = whole.forward(x).clone()
    ids = whole.ids.clone()
    # experts from host memory, all fetched
    layer = bv.MoELayer(s.H, s.I, s.E, s.k, T, lay.codebook, lay.w_router, lay.bias, scoring=how)
    slot = bv.moe_expert_cache_slot_bytes(s.H, s.I, bv.MOE_FMT_VQ2)
    cache = bv.ExpertCache(layer.table, torch.empty(s.E * slot, dtype=torch.uint8, device="cuda"), slot)
    for e in range(s.E):
        cache.set_host_image(e, bv.MOE_FMT_VQ2, bv.host_expert_image(*f(e)))
    assert torch.equal(bv.MissFetchForward(layer, cache, T).step(x), want) and torch.equal(layer.ids, ids)
    # half of the experts on the host
    half, keep2 = bv.upload_layer(s.H, s.I, s.E, s.k, T, lay.codebook, lay.w_router, lay.bias, f, resident=range(4), scoring=how)
    hx = bv.HostExperts(s.E)
    for e in range(4, s.E):
        hx.set(e, *bv.host_pack_expert(*f(e)))
    out = bv.TandemForward(half, bv.CpuPool(2), hx, T).step(x.cpu().pin_memory())
    torch.cuda.synchronize()
    assert torch.equal(half.ids, ids)
    assert_close(out.cpu().numpy(), want.cpu().numpy())
    # a gate without FP4 weights to turn to
    gated = bv.MoELayer(s.H, s.I, s.E, s.k, T, lay.codebook, lay.w_router, lay.bias, table_experts=2 * s.E, scoring=how)
    for e in range(s.E):
        gated.set_expert(e, f(e)[0], *keep[e])
    assert torch.equal(bv.GatedForward(gated, T, tau=0.5).step(x), want)
