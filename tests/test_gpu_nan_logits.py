"""A logit that is NaN makes all of its token's weights NaN, also where its expert is
not among the chosen; other tokens keep theirs."""
import pytest

torch = pytest.importorskip("torch")
import attn_common as ac  # noqa: E402
import rows_common as rc  # noqa: E402
from gpu_common import torch_cuda  # noqa: E402

pytestmark = pytest.mark.gpu

F32 = torch.float32


@pytest.mark.parametrize("E,k,groups,top_groups,group_top", [(8, 2, 1, 1, 1), (64, 8, 1, 1, 1), (64, 8, 8, 4, 2), (257, 5, 1, 1, 1),
                                                             (1024, 32, 32, 8, 2)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renorm", [0, 1])
def test_weights(E, k, groups, top_groups, group_top, sigmoid, biased, renorm):
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    nan = float("nan")
    g = ac.gen(E + k)
    logits = ac.normal(g, 9, E, dtype=F32)
    bias = ac.normal(g, E, dtype=F32, std=0.1) if biased else None
    logits[0] = nan
    logits[1, 1:] = nan
    logits[2, 0] = nan
    logits[3, E - 1] = nan
    logits[4, E // 2] = -nan
    logits[5, int(logits[5].argmin())] = nan
    logits[6, 3] = float("-inf")
    ids = torch.full((9, k), -5, dtype=torch.int32, device="cuda")
    w = torch.zeros(9, k, device="cuda")
    bv.moe_route_scored(logits, k, ids, w, scoring=int(sigmoid), bias=bias, groups=groups, top_groups=top_groups,
                        group_top=group_top, renormalize=renorm, scale=1.5)
    for row in ids.tolist():
        assert len(set(row)) == k and min(row) >= 0 and max(row) < E
    assert bool(torch.isnan(w[:6]).all())
    want, w64 = rc.scored64(logits[6:], k, sigmoid, bias, groups, top_groups, group_top, renorm, 1.5)
    assert torch.equal(ids[6:].cpu(), want)
    # (the tolerance of test_gpu_route_scored.py)
    ac.within(w[6:].cpu(), w64, w64.abs() * 160 * 2.0 ** -23 + 1.5 * 2.0 ** -120, "weights")
    # the whole routing of few tokens too
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    x[0, 0] = x[1, 0] = 1
    wr = torch.zeros(E, 256, dtype=torch.bfloat16, device="cuda")
    wr[E - 1, 5] = nan
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    out = (torch.zeros(2, E, device="cuda"), i32(2, k), torch.zeros(2, k, device="cuda"), i32(E + 1), i32(2 * k), i32(2 * k))
    bv.moe_route_tokens_scored(x, wr, None, k, *out, scoring=int(sigmoid), bias=bias, groups=groups, top_groups=top_groups,
                               group_top=group_top, renormalize=renorm)
    assert bool(torch.isnan(out[2]).all())
