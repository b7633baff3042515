"""moe_router_logits reads tokens and weights that the launch just before writes: the
norm, the logits, the choice by score and the permutation one behind the other."""
import pytest

torch = pytest.importorskip("torch")
import attn_common as ac  # noqa: E402
from gpu_common import torch_cuda  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T", [1, 3, 8, 9, 33, 64, 65])
@pytest.mark.parametrize("H,E", [(512, 8), (4096, 256), (8192, 33)])
def test_tokens_of_the_norm_just_before(T, H, E, graph):
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    n, k = 6, 4
    g = ac.gen(T + H)
    src = [ac.normal(g, T, H, dtype=F32) for _ in range(n)]
    weight, w = ac.normal(g, H), ac.normal(g, E, H, std=0.05)
    rb, bias = ac.normal(g, E, dtype=F32, std=0.1), ac.normal(g, E, dtype=F32, std=0.05)
    x = torch.zeros(T, H, dtype=BF, device="cuda")
    out = [(torch.empty(T, E, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda"),
            torch.empty(T, k, device="cuda")) for _ in range(n)]

    def step(i, o, between=lambda: None):
        bv.moe_rms_norm(src[i], weight, 1e-6, y=x)
        between()
        bv.moe_router_logits(x, w, rb, o[0])
        between()
        bv.moe_route_scored(o[0], k, o[1], o[2], scoring=1, bias=bias)

    step(0, out[0])
    torch.cuda.synchronize()
    if graph:
        c = torch.cuda.CUDAGraph()
        with torch.cuda.graph(c):
            for i in range(n):
                step(i, out[i])
        for _ in range(5):
            c.replay()
    else:
        for _ in range(5):
            for i in range(n):
                step(i, out[i])
    torch.cuda.synchronize()
    for i in range(n):
        want = tuple(torch.empty_like(t) for t in out[i])
        step(i, want, torch.cuda.synchronize)
        assert all(torch.equal(a, b) for a, b in zip(out[i], want)), i


@pytest.mark.parametrize("T", [1, 20])
def test_weights_of_the_call_just_before(T):
    """The router's weights too may come from the launch ahead."""
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    H, E = 1024, 64
    g = ac.gen(T)
    x, src = ac.normal(g, T, H), [ac.normal(g, E, H, dtype=F32) for _ in range(4)]
    w = torch.zeros(E, H, dtype=BF, device="cuda")
    out = [torch.empty(T, E, device="cuda") for _ in src]
    for _ in range(5):
        for s, o in zip(src, out):
            bv.moe_rms_norm(s, None, 1e-6, y=w)
            bv.moe_router_logits(x, w, None, o)
    torch.cuda.synchronize()
    for s, o in zip(src, out):
        bv.moe_rms_norm(s, None, 1e-6, y=w)
        torch.cuda.synchronize()
        want = torch.empty_like(o)
        bv.moe_router_logits(x, w, None, want)
        assert torch.equal(o, want)
