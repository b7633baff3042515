"""moe_linear behind the work that writes its operands: weights, bias, tokens
and residual written by the launch just before the call, by another library's
kernel and by a moe_linear, eagerly and in a captured graph."""
import pytest

from gpu_common import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T", [1, 8, 9, 32, 64, 128, 300])
def test_operands_written_just_before(T, graph):
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    K, N, n = 4096, 1024, 6
    g = ac.gen(T)
    x, b, r = ac.normal(g, T, K), ac.normal(g, N), ac.normal(g, T, N)
    ws_ = [ac.normal(g, N, K, std=K ** -0.5) for _ in range(n)]
    w = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    bias, res = torch.zeros_like(b), torch.zeros_like(r)
    ys = torch.empty(n, T, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(bv.moe_linear_workspace_size(T, N, K), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()

    def steps():
        for i in range(n):
            res.copy_(r)
            bias.copy_(b)
            torch.mul(ws_[i], 1.0, out=w)
            bv.moe_linear(x, w, ys[i], bias, bv.MOE_ACT_NONE, res, ws)

    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        if graph:
            c = torch.cuda.CUDAGraph()
            with torch.cuda.graph(c, stream=stream):
                steps()
            for _ in range(5):
                c.replay()
        else:
            for _ in range(5):
                steps()
    torch.cuda.synchronize()
    for i in range(n):
        want, tol = ac.linear64(x, ws_[i], b, 0, r)
        ac.within(ys[i], want, tol, f"step {i}")
    assert int(ws[8:12].view(torch.int32).item()) == 0


@pytest.mark.parametrize("T", [1, 32, 300])
def test_weights_from_a_product(T):
    # w is the result of a moe_linear just before
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    K, N, R = 2048, 512, 64
    g = ac.gen(T)
    x = ac.normal(g, T, K)
    w, y = (torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in ((N, K), (T, N)))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for i in range(10):
        up, down = ac.normal(g, N, R), ac.normal(g, K, R, std=(R * K) ** -0.5)
        bv.moe_linear(up, down, w, ws=ws)
        bv.moe_linear(x, w, y, ws=ws)
        want, tol = ac.linear64(x, w, None, 0, None)
        ac.within(y, want, tol, f"product {i}")
        wp, tp = ac.linear64(up, down, None, 0, None)
        ac.within(w, wp, tp, f"weights of product {i}")
