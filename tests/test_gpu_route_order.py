"""moe_route_fresh: moe_route's results, for tokens that the launch just before
writes -- a torch kernel or a moe_linear -- eagerly and in a captured graph."""
import pytest

import moe_synth as ms
from gpu_common import device_layer, torch_cuda

pytestmark = pytest.mark.gpu

T_MAX = 40


@pytest.fixture(scope="module")
def dev():
    torch_cuda()
    layer, keep = device_layer(ms.Layer(ms.spec_tiny(0)), T_MAX)
    yield layer
    del keep


def _routed(dev, T):
    P = T * dev.k
    return [t.clone() for t in (dev.logits[:T], dev.ids[:T], dev.weights[:T], dev.offsets, dev.sorted_pair[:P],
                                dev.pair_to_sorted[:P])]


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 40])
def test_same_bits(dev, T):
    torch = torch_cuda()
    import attn_common as ac
    x = ac.normal(ac.gen(T), T, dev.H)
    dev.route(x)
    want = _routed(dev, T)
    dev.route(x, fresh=True)
    assert all(torch.equal(a, b) for a, b in zip(_routed(dev, T), want))


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("writer", ["torch", "linear"])
@pytest.mark.parametrize("T", [1, 4, 40])
def test_tokens_written_just_before(dev, T, writer, graph):
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    n, H = 8, dev.H
    g = ac.gen(T)
    src = [ac.normal(g, T, H) for _ in range(n)]
    w = ac.normal(g, H, H, std=H ** -0.5)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    logits = torch.empty(n, T, dev.w_router.shape[0], device="cuda")
    outs = torch.empty(n, T, H, device="cuda")

    def write(i):
        if writer == "torch":
            torch.mul(src[i], 1.0, out=x)
        else:
            bv.moe_linear(src[i], w, x, ws=ws)

    def steps():
        for i in range(n):
            write(i)
            dev.forward(x, out=outs[i], fresh=True)
            logits[i].copy_(dev.logits[:T])

    write(0)
    dev.forward(x, out=outs[0], fresh=True)  # (kernel attributes are set outside capture)
    torch.cuda.synchronize()
    if graph:
        c = torch.cuda.CUDAGraph()
        with torch.cuda.graph(c):
            steps()
        for _ in range(5):
            c.replay()
    else:
        for _ in range(5):
            steps()
    torch.cuda.synchronize()
    for i in range(n):
        write(i)
        torch.cuda.synchronize()
        y = dev.forward(x)
        torch.cuda.synchronize()
        assert torch.equal(logits[i], dev.logits[:T]) and torch.equal(outs[i], y), i
