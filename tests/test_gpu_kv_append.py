"""moe_kv_append against 64 bits: both rotations, partial and no rotation,
both cache orders, slices of one projection's rows, padding, tokens that the
device has to keep from harm."""
import math

import pytest

from gpu_common import torch_cuda

pytestmark = pytest.mark.gpu


def _table(torch, n, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float()


def _turn64(torch, x, cs, rot, inter):
    x = x.double().clone()
    c, s = cs[:, None, :rot // 2].double(), cs[:, None, rot // 2:].double()
    ia = torch.arange(0, rot, 2) if inter else torch.arange(rot // 2)
    ib = ia + 1 if inter else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


def _case(T, heads, group, D, rot, inter, page, dtype, order="token", skip=0, seed=0, in_place=False, with_q=True):
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    dt = getattr(torch, dtype)
    g = ac.gen(seed)
    qkv = ac.normal(g, T, (group + 2) * heads, D, dtype=dt)
    orig = qkv.clone()
    q, k, v = qkv[:, :group * heads], qkv[:, group * heads:(group + 1) * heads], qkv[:, (group + 1) * heads:]
    oq, ok, ov = orig[:, :group * heads], orig[:, group * heads:(group + 1) * heads], orig[:, (group + 1) * heads:]
    pages = -(-T // page) + 2
    shape = (pages, page, heads, D) if order == "token" else (pages, heads, page, D)
    kc, vc = ac.normal(g, *shape, dtype=dt), ac.normal(g, *shape, dtype=dt)
    kv, vv = (kc, vc) if order == "token" else (kc.transpose(1, 2), vc.transpose(1, 2))
    wk, wv = kv.double().clone(), vv.double().clone()
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    if skip:
        slots[::skip] = -1 - torch.arange(0, T, skip, device="cuda")
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=torch.int32)
    cs = _table(torch, 5000, rot) if rot else None
    qo = q if in_place else torch.full_like(q, 3.0)
    kw = dict(q=q, q_out=qo) if with_q else {}
    bv.moe_kv_append(k, v, kv, vv, pos, slots, cs, interleaved=inter, **kw)
    tq = _turn64(torch, oq, cs[pos.long()], rot, inter) if rot else oq.double()
    tk = _turn64(torch, ok, cs[pos.long()], rot, inter) if rot else ok.double()
    t = torch.nonzero(slots >= 0).flatten()
    wk[slots[t] // page, slots[t] % page] = tk[t]
    wv[slots[t] // page, slots[t] % page] = ov[t].double()
    # two products and a sum in fp32 (3 e of |a| + |b| <= sqrt 2 |(a, b)|), one rounding
    u = ac.U[dt]

    def tol(x):
        n = (x.double() ** 2).sum(-1, keepdim=True).sqrt()
        return u * x.abs() + 4 * ac.E23 * n + ac.TINY[dt]

    if with_q:
        ac.within(qo, tq, tol(tq), "q")
        if rot < D:
            assert torch.equal(qo[..., rot:], oq[..., rot:])
    ac.within(kv, wk, tol(wk), "k")
    assert torch.equal(vv.double(), wv)
    # slots that were not named keep their bits
    named = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
    named[slots[t]] = True
    assert torch.equal(kv.reshape(-1, heads, D)[~named].double(), wk.reshape(-1, heads, D)[~named])


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (80, 32), (64, 64), (8, 0), (24, 16), (72, 48), (256, 256), (80, 40), (96, 24), (64, 12),
                                   (128, 36), (64, 6), (80, 2), (8, 8), (200, 100)])
def test_head_sizes(D, rot, inter, dtype):
    _case(37, 2, 3, D, rot, inter, 16, dtype, seed=D + rot)


@pytest.mark.parametrize("T", [1, 2, 31, 600])
@pytest.mark.parametrize("heads,group", [(1, 1), (8, 4), (3, 5), (1, 40)])
def test_tokens_and_heads(T, heads, group):
    _case(T, heads, group, 128, 128, False, 32, "bfloat16", seed=T)


@pytest.mark.parametrize("page", [1, 3, 16, 100])
@pytest.mark.parametrize("order", ["token", "head"])
def test_pages_and_cache_orders(page, order):
    _case(65, 4, 2, 64, 64, True, page, "float16", order, skip=5, seed=page)


def test_in_place_and_keys_only():
    _case(50, 2, 4, 128, 128, False, 16, "bfloat16", in_place=True)
    _case(50, 2, 4, 128, 64, True, 16, "bfloat16", in_place=True)
    _case(50, 2, 4, 128, 128, False, 16, "bfloat16", with_q=False)


def test_slots_and_positions_out_of_range_do_no_harm():
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    g = ac.gen(3)
    T, heads, D = 6, 2, 64
    k, v, q = (ac.normal(g, T, heads, D) for _ in range(3))
    kc, vc = torch.zeros(3, 8, heads, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 8, heads, D,
                                                                                          dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, 24, 1 << 40, -(1 << 40), 5, 6], device="cuda")
    pos = torch.tensor([1, 1, 1, 1, 100, -1], dtype=torch.int32, device="cuda")
    qo = torch.zeros_like(q)
    bv.moe_kv_append(k, v, kc, vc, pos, slots, _table(torch, 100, D), q=q, q_out=qo)
    written = torch.nonzero(vc.reshape(24, -1).any(1)).flatten().tolist()
    assert written == [0] and torch.nonzero(kc.reshape(24, -1).any(1)).flatten().tolist() == [0]
    assert bool(torch.isfinite(qo[:4]).all()) and bool(torch.isnan(qo[4:]).all())
    assert math.isfinite(float(kc.float().sum()))


def test_offsets_past_32_bits():
    # keys and values of over 2^32 elements each
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    heads, D, page = 8, 128, 64
    pages = 2 ** 32 // (heads * D * page) + 2
    kc = torch.empty(pages, page, heads, D, dtype=torch.bfloat16, device="cuda")
    g = ac.gen(5)
    k, v = ac.normal(g, 2, heads, D), ac.normal(g, 2, heads, D)
    slots = torch.tensor([pages * page - 1, 3], device="cuda")
    vc = torch.empty_like(kc)
    bv.moe_kv_append(k, v, kc, vc, None, slots)
    assert torch.equal(kc[-1, -1], k[0]) and torch.equal(kc[0, 3], k[1])
    assert torch.equal(vc[-1, -1], v[0]) and torch.equal(vc[0, 3], v[1])
