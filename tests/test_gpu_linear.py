"""moe_linear against 64 bits: every activation, both types, token counts on
both sides of every tile size, odd output counts, strided rows, in-place
residual, other streams, graphs."""
import pytest

from gpu_common import torch_cuda

pytestmark = pytest.mark.gpu

TYPES = ["bfloat16", "float16"]


def _run(T, K, N, dtype, act=0, bias=False, residual=False, padx=0, padw=0, pady=0, seed=0, big=False):
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    dt = getattr(torch, dtype)
    g = ac.gen(seed)
    x = ac.normal(g, T, K + padx, dtype=dt)[:, :K]
    w = ac.normal(g, N, K + padw, dtype=dt, std=K ** -0.5)[:, :K]
    b = ac.normal(g, N, dtype=dt) if bias else None
    r = ac.normal(g, T, N + 3, dtype=dt, std=4.0)[:, 1:N + 1] if residual else None
    hold = torch.full((T + 2, N + pady), 7.0, dtype=dt, device="cuda")
    y = hold[1:T + 1, :N]
    ws = torch.zeros(bv.moe_linear_workspace_size(T, N, K), dtype=torch.uint8, device="cuda")
    bv.moe_linear(x, w, y, bias=b, act=act, residual=r, ws=ws)
    want, tol = ac.linear64(x, w, b, act, r)
    ac.within(y, want, tol, f"T={T} K={K} N={N}")
    # nothing outside y
    assert bool((hold[0] == 7).all()) and bool((hold[-1] == 7).all()) and bool((hold[:, N:] == 7).all())
    assert int(ws[8:12].view(torch.int32).item()) == 0
    first = y.clone()
    bv.moe_linear(x, w, y, bias=b, act=act, residual=r, ws=ws)
    assert torch.equal(y, first)  # the same sums in the same order, whatever ran before


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 32, 33, 64, 65, 100, 128, 129, 200, 256, 257, 300, 513])
def test_token_counts(T, dtype):
    _run(T, 520, 391, dtype, bias=True, seed=T)


@pytest.mark.parametrize("N", [1, 2, 7, 63, 64, 65, 127, 128, 129, 255, 257, 1000])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_output_counts(T, N):
    _run(T, 256, N, "bfloat16", residual=True, pady=1, seed=N)


@pytest.mark.parametrize("K", [8, 16, 24, 56, 64, 72, 128, 136, 1000, 4096, 8192])
@pytest.mark.parametrize("T", [1, 33, 270])
def test_sum_lengths(T, K):
    _run(T, K, 200, "float16", bias=True, seed=K)


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("T", [3, 150])
@pytest.mark.parametrize("dtype", TYPES)
def test_activations(act, T, dtype):
    _run(T, 192, 130, dtype, act, True, True, seed=act)


@pytest.mark.parametrize("T", [1, 20, 300])
def test_strided_rows(T):
    _run(T, 264, 333, "bfloat16", 4, True, True, 24, 8, 5, seed=9)


@pytest.mark.parametrize("T", [1, 32, 500])
def test_many_output_tiles(T):
    _run(T, 64, 20011, "bfloat16", bias=True, seed=11)


def test_residual_in_place():
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    for T in (1, 30, 400):
        g = ac.gen(T)
        x, w = ac.normal(g, T, 512), ac.normal(g, 384, 512, std=0.05)
        y = ac.normal(g, T, 384)
        ws = torch.zeros(bv.moe_linear_workspace_size(T, 384, 512), dtype=torch.uint8, device="cuda")
        want, tol = ac.linear64(x, w, None, 0, y.clone())
        bv.moe_linear(x, w, y, residual=y, ws=ws)
        ac.within(y, want, tol, f"T={T}")


def test_infinities_and_nan_stay_in_their_rows_and_columns():
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    for T in (5, 200):
        g = ac.gen(1)
        x, w = ac.normal(g, T, 128), ac.normal(g, 140, 128)
        x[3, 5] = float("nan")
        w[77, 9] = float("inf")
        y = torch.empty(T, 140, dtype=torch.bfloat16, device="cuda")
        ws = torch.zeros(bv.moe_linear_workspace_size(T, 140, 128), dtype=torch.uint8, device="cuda")
        bv.moe_linear(x, w, y, ws=ws)
        assert bool(torch.isnan(y[3]).all())
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[3] = False
        cols = torch.arange(140, device="cuda") != 77
        assert bool(torch.isfinite(y[keep][:, cols]).all())
        assert not bool(torch.isfinite(y[:, 77]).any())


def test_other_stream_and_graph():
    torch = torch_cuda()
    import attn_common as ac
    import bit_vq_routed_gb300 as bv
    g = ac.gen(4)
    x, w = ac.normal(g, 24, 1024), ac.normal(g, 500, 1024, std=0.03)
    want, tol = ac.linear64(x, w, None, 0, None)
    y = torch.empty(24, 500, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(bv.moe_linear_workspace_size(24, 500, 1024), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bv.moe_linear(x, w, y, ws=ws)
    s.synchronize()
    ac.within(y, want, tol, "side stream")
    y.zero_()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        bv.moe_linear(x, w, y, ws=ws)
    x.mul_(2)
    gr.replay()
    want, tol = ac.linear64(x, w, None, 0, None)
    ac.within(y, want, tol, "graph replay on new inputs")


def test_empty_calls_launch_nothing():
    torch = torch_cuda()
    import bit_vq_routed_gb300 as bv
    n = bv.moe_launch_count()
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(8, 64, dtype=torch.bfloat16, device="cuda")
    bv.moe_linear(x, w, torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"))
    assert bv.moe_launch_count() == n
