"""moe_prefix_attention with more sequences than a CTA keeps in shared memory
(512) and with more units of work than one launch takes (2048), where a call is
cut at a token and sequences lie across the cut."""
import math

import pytest

from gpu_common import torch_cuda
from test_gpu_prefix_attention import _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [511, 512, 513, 700])
@pytest.mark.parametrize("prefix", [0, 200])
def test_many_sequences(B, prefix):
    # 0 to 2 new tokens each, some sequences without any of their own
    nq = [(0, 1, 1, 2)[i % 4] for i in range(B)]
    lens = [max(n, 7 * i % 60) if i % 11 else n for i, n in enumerate(nq)]
    _check(_inputs(nq, lens, prefix, 1, 4, 64, 8, seed=B))


def test_many_sequences_in_pairs_of_tiles():
    nq = [(0, 9, 5, 40)[i % 4] for i in range(600)]
    _check(_inputs(nq, [n + 13 * i % 90 for i, n in enumerate(nq)], 130, 1, 4, 64, 16, "float16", seed=1))


@pytest.mark.parametrize("nq,lead", [([2000, 1500, 0, 700, 900], 0), ([4090, 1, 5, 3, 800], 0), ([4096, 900], 0),
                                     ([1000, 3500], 3)])
def test_more_units_than_one_launch(nq, lead):
    # 128 query heads to the key head: a tile holds one token, a launch 4096
    _check(_inputs(nq, [n + 40 * i for i, n in enumerate(nq)], 70, 1, 128, 16, 16, seed=2, lead=lead))


def test_more_units_than_one_launch_of_single_tokens():
    # 16 tokens to a tile, single tiles (few rows a sequence): 32768 tokens a launch
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    B, G, D, page, prefix = 33000, 8, 32, 8, 21
    g = ac.gen(3)
    kc, vc = (ac.normal(g, B + 3, page, 1, D) for _ in range(2))
    q = ac.normal(g, B, G, D, std=2.0)
    perm = torch.randperm(B + 3, generator=g, device="cuda").to(torch.int32)
    lens = torch.randint(0, page + 1, (B,), generator=g, device="cuda").to(torch.int32)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    table = perm[3:, None].contiguous()
    out, lse = torch.full_like(q, 7.0), torch.full((B, G), 7.0, device="cuda")
    ws = torch.zeros(bv.moe_prefix_attention_workspace_size(B, G, 1, D), dtype=torch.uint8, device="cuda")
    n = bv.moe_launch_count()
    bv.moe_prefix_attention(q, kc, vc, cu, perm[:3], prefix, table, lens, 0.25, out, lse, ws)
    assert bv.moe_launch_count() - n == 4  # (two kernels, twice)
    assert int(ws[8:12].view(torch.int32).item()) == 0
    shared = [c[perm[:3].long()].reshape(-1, D)[:prefix].double().expand(B, prefix, D) for c in (kc, vc)]
    K, V = (torch.cat((s, c[table[:, 0].long()].view(B, page, D).double()), 1) for s, c in zip(shared, (kc, vc)))
    S = 0.25 * torch.einsum("bgd,bkd->bgk", q.double(), K)
    mag = 0.25 * torch.einsum("bgd,bkd->bgk", q.double().abs(), K.abs())
    hidden = (torch.arange(prefix + page, device="cuda") >= prefix + lens[:, None])[:, None]
    S, mag = S.masked_fill(hidden, -math.inf), mag.masked_fill(hidden, 0.0)
    P = torch.softmax(S, -1)
    o, A, N, u = P @ V, P @ V.abs(), prefix + page + 8, ac.U[q.dtype]
    # (the arithmetic of attention64's tolerance)
    d = (D + 4) * ac.E23 * mag.amax(-1, keepdim=True) + 2.0 ** -21
    ac.within(out, o, (u + torch.expm1(4 * d) + 4 * N * ac.E23) * (1 + u) * A + u * o.abs(), "out")
    l = torch.logsumexp(S, -1)
    ac.within(lse, l, d[..., 0] + 2 * N * ac.E23 + 4 * ac.E23 * l.abs(), "lse")
