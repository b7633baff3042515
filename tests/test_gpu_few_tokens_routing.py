"""moe_route_tokens_scored: up to 8 tokens of 5120 logits in all the choice and the
permutation are one kernel; the results are the three steps' on both sides."""
import pytest

torch = pytest.importorskip("torch")
import attn_common as ac  # noqa: E402
from gpu_common import torch_cuda  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k,groups", [(8, 2, 1), (60, 7, 1), (256, 8, 8), (640, 32, 16), (641, 5, 1), (736, 8, 32), (1000, 31, 20),
                                        (1024, 32, 1), (1024, 8, 32)])
@pytest.mark.parametrize("T", [1, 5, 6, 7, 8, 9])
def test_launches_and_results(T, E, k, groups):
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    g = ac.gen(T + E)
    H = 256
    x, w = ac.normal(g, T, H), ac.normal(g, E, H, std=0.1)
    bias = ac.normal(g, E, dtype=torch.float32, std=0.05)
    how = dict(scoring=1, bias=bias, groups=groups, top_groups=(groups + 1) // 2, group_top=2 if groups > 1 else 1)
    i32 = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")  # noqa: E731
    outs = lambda: (torch.zeros(T, E, device="cuda"), i32(T, k), torch.zeros(T, k, device="cuda"),  # noqa: E731
                    i32(E + 1), i32(T * k), i32(T * k))
    a, b = outs(), outs()
    n = bv.moe_launch_count()
    bv.moe_route_tokens_scored(x, w, None, k, *a, **how)
    assert bv.moe_launch_count() - n == (2 if T <= 8 and T * (E + E % 2) <= 5120 else 3)
    bv.moe_router_logits(x, w, None, b[0])
    bv.moe_route_scored(b[0], k, b[1], b[2], **how)
    bv.moe_permute(b[1], E, *b[3:])
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    # captured, from the first call of its size on
    c = torch.cuda.CUDAGraph()
    with torch.cuda.graph(c):
        bv.moe_route_tokens_scored(x, w, None, k, *a, **how)
    x.copy_(ac.normal(g, T, H))
    c.replay()
    bv.moe_router_logits(x, w, None, b[0])
    bv.moe_route_scored(b[0], k, b[1], b[2], **how)
    bv.moe_permute(b[1], E, *b[3:])
    assert all(torch.equal(p, q) for p, q in zip(a, b))
