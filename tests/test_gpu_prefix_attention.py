"""moe_prefix_attention against 64 bits: single tokens and prompts, ragged
batches, empty sequences and empty rows, pages that end inside a tile, both
cache orders, and a cache whose unused slots hold NaN."""
import pytest

from gpu_common import torch_cuda

pytestmark = pytest.mark.gpu


def _inputs(nq, lens, prefix, heads, group, D, page, dtype="bfloat16", order="token", seed=0, lead=0, trail=0, std=2.0):
    torch = torch_cuda()
    import attn_common as ac
    dt = getattr(torch, dtype)
    g = ac.gen(seed)
    B, T = len(nq), sum(nq) + lead + trail
    shared, each = -(-prefix // page), [-(-m // page) for m in lens]
    pages = shared + sum(each) + 3
    shape = (pages, page, heads, D) if order == "token" else (pages, heads, page, D)
    kc, vc = ac.normal(g, *shape, dtype=dt), ac.normal(g, *shape, dtype=dt)
    if order == "head":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    order_ = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(each + [1]) + 2), -5, dtype=torch.int32, device="cuda")
    used = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    pp = order_[:shared].contiguous()
    used[pp.long()] = True
    if prefix % page:
        used[int(pp[-1]), prefix % page:] = False
    at = shared
    for b, n in enumerate(each):
        ids = order_[at:at + n]
        table[b, :n] = ids
        used[ids.long()] = True
        if lens[b] % page:
            used[int(ids[-1]), lens[b] % page:] = False
        at += n
    kc[~used] = float("nan")  # (what no sequence holds must not reach a result)
    vc[~used] = float("nan")
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(nq, dtype=torch.int32).cumsum(0)
    cu += lead
    q = ac.normal(g, T, heads * group, D, dtype=dt, std=std)
    return dict(q=q, k_cache=kc, v_cache=vc, cu_q=cu.cuda(), prefix_pages=pp, prefix_len=prefix, page_table=table,
                seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=D ** -0.5)


def _check(a, want_lse=True, ws=None, what=""):
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    q = a["q"]
    T, Hq, D = q.shape
    heads = a["k_cache"].shape[2]
    hold = torch.full((T + 2, Hq, D), 7.0, dtype=q.dtype, device="cuda")
    out = hold[1:-1]
    lse = torch.full((T, Hq), 7.0, device="cuda") if want_lse else None
    if ws is None:
        ws = torch.zeros(bv.moe_prefix_attention_workspace_size(T, Hq, heads, D), dtype=torch.uint8, device="cuda")
    bv.moe_prefix_attention(**a, out=out, lse=lse, ws=ws)
    wo, wl, to, tl = ac.attention64(q, a["k_cache"], a["v_cache"], a["cu_q"], a["prefix_pages"], a["prefix_len"],
                                    a["page_table"], a["seq_lens"], a["scale"])
    ac.within(out, wo, to, what + " out")
    if want_lse:
        assert torch.equal(torch.isinf(lse), torch.isinf(wl)) and bool((lse[torch.isinf(lse)] < 0).all())
        f = torch.isfinite(wl)
        ac.within(lse[f], wl[f], tl[f], what + " lse")
    assert bool((hold[0] == 7).all()) and bool((hold[-1] == 7).all())
    assert int(ws[8:12].view(torch.int32).item()) == 0
    first = (out.clone(), None if lse is None else lse.clone())
    bv.moe_prefix_attention(**a, out=out, lse=lse, ws=ws)  # (a used workspace; the same bits again)
    assert torch.equal(out, first[0]) and (lse is None or torch.equal(lse, first[1]))


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000, 5000])
@pytest.mark.parametrize("own", [1, 100, 300])
def test_single_token(prefix, own):
    _check(_inputs([1], [own], prefix, 2, 4, 128, 16, seed=prefix + own))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("D", [8, 16, 24, 40, 64, 72, 80, 96, 104, 120, 128])
def test_head_sizes(D, dtype):
    _check(_inputs([1, 5, 40], [30, 5, 200], 77, 2, 3, D, 16, dtype, seed=D))


@pytest.mark.parametrize("heads,group", [(1, 1), (8, 1), (1, 7), (5, 3), (2, 16), (1, 33), (1, 64), (1, 100), (1, 128)])
def test_head_layouts(heads, group):
    _check(_inputs([1, 3, 0, 20], [9, 3, 4, 150], 130, heads, group, 64, 32, seed=group))


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("order", ["token", "head"])
def test_page_sizes_and_cache_orders(page, order):
    _check(_inputs([1, 1, 60, 1], [1, page, page + 60, 3 * page - 1], 2 * page + 3, 2, 4, 80, page, order=order, seed=page))


def test_batch_of_single_tokens():
    g = [1 + (37 * i) % 500 for i in range(64)]
    _check(_inputs([1] * 64, g, 2049, 2, 8, 128, 64, seed=1))
    _check(_inputs([1] * 200, [1 + i % 9 for i in range(200)], 300, 1, 4, 64, 8, seed=2))


@pytest.mark.parametrize("nq", [127, 128, 129, 400])
@pytest.mark.parametrize("prefix", [0, 200])
def test_prompts(nq, prefix):
    _check(_inputs([nq], [nq], prefix, 2, 2, 128, 16, seed=nq))
    _check(_inputs([nq, 3, nq // 2], [nq + 70, 3, nq], prefix, 1, 4, 64, 64, "float16", seed=nq))


def test_many_rows_and_few():
    # a prompt of one sequence beside single tokens of others
    _check(_inputs([600] + [1] * 20, [900] + [10 * i + 1 for i in range(20)], 513, 2, 4, 128, 16, seed=3))


def test_long_single_sequence():
    _check(_inputs([1], [20000], 0, 1, 8, 128, 16, seed=4))
    _check(_inputs([2, 1], [10000, 3], 30000, 1, 4, 128, 128, seed=5))


def test_rows_that_see_nothing():
    # no prefix, and more query tokens than cached ones: the first rows are empty
    _check(_inputs([10, 4, 1], [3, 0, 0], 0, 2, 2, 64, 16, seed=6), what="empty rows")
    _check(_inputs([300, 200], [50, 0], 0, 1, 4, 128, 16, seed=7), what="empty tiles")
    _check(_inputs([10, 4], [3, 0], 20, 2, 2, 64, 16, seed=8), what="prefix only")


def test_tokens_of_no_sequence():
    _check(_inputs([1, 5], [20, 30], 40, 2, 2, 64, 16, seed=9, lead=3, trail=2))
    _check(_inputs([0, 0], [20, 30], 40, 2, 2, 64, 16, seed=10, lead=3, trail=200))


def test_large_scores_and_no_lse():
    # scores of several hundred: one key takes all the weight, the running maximum jumps
    _check(_inputs([1, 70], [300, 500], 700, 2, 4, 128, 16, seed=11, std=60.0))
    _check(_inputs([1, 70], [300, 500], 700, 2, 4, 128, 16, "float16", seed=12, std=30.0), want_lse=False)


def test_rising_and_falling_scores():
    # keys whose scores rise along the sequence (every tile brings a new maximum), then fall
    torch = torch_cuda()
    for sign in (1, -1):
        a = _inputs([1, 40], [800, 900], 1500, 1, 4, 64, 16, seed=13)
        a["q"][:] = 0.5
        ids = a["prefix_pages"].long()
        ramp = torch.linspace(-1, 1, 1504, device="cuda") * sign
        a["k_cache"][ids] = (ramp.view(-1, 16, 1, 1) * 6).to(torch.bfloat16)
        _check(a)


def test_lengths_past_the_table_are_cut():
    torch = torch_cuda()
    a = _inputs([1, 2], [40, 33], 20, 2, 2, 64, 16, seed=14)
    a["page_table"] = a["page_table"][:, :3]
    ids = a["page_table"][0].long()
    for c in ("k_cache", "v_cache"):
        a[c][ids] = a[c][ids].nan_to_num(0.5)
    a["seq_lens"] = torch.tensor([1 << 30, 33], dtype=torch.int32, device="cuda")
    _check(a)


def test_workspace_shared_by_calls_of_several_shapes():
    torch = torch_cuda()
    import bit_vq_routed_gb300 as bv
    cases = [_inputs([1] * 8, [100 * i + 1 for i in range(8)], 3000, 2, 4, 128, 64, seed=15),
             _inputs([300], [300], 100, 2, 4, 128, 64, seed=16), _inputs([1], [5], 3, 2, 4, 128, 64, seed=17)]
    n = max(bv.moe_prefix_attention_workspace_size(c["q"].shape[0], 8, 2, 128) for c in cases)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for c in cases + cases[::-1]:
        _check(c, ws=ws)


def test_graph_follows_lengths():
    # a captured call reads the lengths and pages of each replay
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    a = _inputs([1] * 4, [50, 60, 70, 80], 333, 2, 4, 128, 16, seed=18)
    out = torch.empty_like(a["q"])
    ws = torch.zeros(bv.moe_prefix_attention_workspace_size(4, 8, 2, 128), dtype=torch.uint8, device="cuda")
    bv.moe_prefix_attention(**a, out=out, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bv.moe_prefix_attention(**a, out=out, ws=ws)
    for lens in ([1, 1, 1, 1], [50, 3, 70, 0], [17, 60, 16, 80]):
        a["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        wo, _, to, _ = ac.attention64(a["q"], a["k_cache"], a["v_cache"], a["cu_q"], a["prefix_pages"], 333,
                                      a["page_table"], a["seq_lens"], a["scale"])
        ac.within(out, wo, to, str(lens))


def test_strided_queries_and_outputs():
    torch = torch_cuda()
    a = _inputs([1, 50], [20, 90], 100, 2, 4, 64, 16, seed=19)
    wide = torch.zeros(51, 13, 72, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:11, :64] = a["q"]
    a["q"] = wide[:, 3:11, :64]
    _check(a)


def _poison(a, b, key, value, page):
    """Sets component 3 of the values of sequence b's own token `key`."""
    p = int(a["page_table"][b, key // page])
    a["v_cache"][p, key % page, :, 3] = value


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("shape", ["tokens", "prompt", "mixed"])
def test_what_is_not_finite_stays_with_its_sequence(shape, value):
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    nq, lens, key = {"tokens": ([1] * 40, [60 + 9 * i for i in range(40)], 55), "prompt": ([700, 30], [700, 30], 333),
                     "mixed": ([50, 1, 90, 1], [200, 300, 90, 7], 170)}[shape]
    a = _inputs(nq, lens, 300, 2, 4, 128, 16, seed=31)
    want, wl, tol, _ = ac.attention64(a["q"], a["k_cache"], a["v_cache"], a["cu_q"], a["prefix_pages"], 300,
                                      a["page_table"], a["seq_lens"], a["scale"])
    b = 0 if shape != "tokens" else 7
    _poison(a, b, key, value, 16)
    out = torch.empty_like(a["q"])
    ws = torch.zeros(bv.moe_prefix_attention_workspace_size(out.shape[0], 8, 2, 128), dtype=torch.uint8, device="cuda")
    for _ in range(5):
        bv.moe_prefix_attention(**a, out=out, ws=ws)
        # of sequence b, the queries that see the key: not finite; every other one as before
        cu = a["cu_q"].tolist()
        hit = torch.zeros(out.shape[0], dtype=torch.bool, device="cuda")
        for t in range(cu[b], cu[b + 1]):
            hit[t] = key <= lens[b] - (cu[b + 1] - 1 - t) - 1
        assert bool(hit.any())
        assert not bool(torch.isfinite(out[hit][..., 3]).any())
        ac.within(out[~hit], want[~hit], tol[~hit], shape)


def test_keys_that_are_not_finite_stay_with_their_sequence():
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    a = _inputs([1] * 20, [70] * 20, 200, 2, 4, 64, 16, seed=32)
    want, _, tol, _ = ac.attention64(a["q"], a["k_cache"], a["v_cache"], a["cu_q"], a["prefix_pages"], 200,
                                     a["page_table"], a["seq_lens"], a["scale"])
    a["k_cache"][int(a["page_table"][4, 2]), 5, :, 7] = float("nan")
    out = torch.empty_like(a["q"])
    ws = torch.zeros(bv.moe_prefix_attention_workspace_size(20, 8, 2, 64), dtype=torch.uint8, device="cuda")
    bv.moe_prefix_attention(**a, out=out, ws=ws)
    keep = torch.arange(20, device="cuda") != 4
    assert bool(torch.isnan(out[4]).all())
    ac.within(out[keep], want[keep], tol[keep], "others")


@pytest.mark.parametrize("heads,group,D,page", [(2, 4, 128, 16), (1, 3, 80, 8), (2, 16, 64, 128), (1, 128, 40, 32)])
@pytest.mark.parametrize("prefix", [0, 700])
def test_many_sequences_in_pairs_of_tiles(heads, group, D, page, prefix):
    # over a thousand rows of a head, tiles shared by sequences of 0 to 40 tokens
    nq = [11 * i % 41 for i in range(30)]
    lens = [max(0, n + (37 * i) % 300 - 20) for i, n in enumerate(nq)]
    _check(_inputs(nq, lens, prefix, heads, group, D, page, seed=33, lead=2, trail=3))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_with_its_sequence_in_pairs_of_tiles(value):
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    nq, lens = [20] * 24, [20 + 31 * i % 300 for i in range(24)]
    a = _inputs(nq, lens, 150, 2, 4, 128, 16, seed=34)
    want, _, tol, _ = ac.attention64(a["q"], a["k_cache"], a["v_cache"], a["cu_q"], a["prefix_pages"], 150,
                                     a["page_table"], a["seq_lens"], a["scale"])
    hit = torch.zeros(sum(nq), dtype=torch.bool, device="cuda")
    for b, back in ((0, 7), (5, 1), (9, 19), (23, 12)):  # the key `back` tokens before the last
        key = lens[b] - 1 - back
        _poison(a, b, key, value, 16)
        hit[sum(nq[:b + 1]) - 1 - back:sum(nq[:b + 1])] = True
    out = torch.empty_like(a["q"])
    ws = torch.zeros(bv.moe_prefix_attention_workspace_size(sum(nq), 8, 2, 128), dtype=torch.uint8, device="cuda")
    for _ in range(5):
        bv.moe_prefix_attention(**a, out=out, ws=ws)
        assert not bool(torch.isfinite(out[hit][..., 3]).any())
        ac.within(out[~hit], want[~hit], tol[~hit], "others")
