"""moe_linear_8bit against 64 bits: each of its kernels (few tokens, split,
pairs), odd sizes, strides, epilogues."""
import pytest

torch = pytest.importorskip("torch")
import attn_common as ac  # noqa: E402
import rows_common as rc  # noqa: E402
from gpu_common import torch_cuda  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16


def _rows(g, T, K, pad=0, std=1.0):
    """8-bit rows of a spread of sizes, and their scales."""
    v = torch.randn(T, K, generator=g, device="cuda") * torch.exp(0.7 * torch.randn(T, 1, generator=g, device="cuda")) * std
    a = v.abs().amax(1, keepdim=True)
    return rc.wide((v * 448 / a).to(rc.E4M3), pad), a[:, 0] / 448


def _run(T, N, K, dt=BF, act=0, bias=False, residual=False, pad=0, seed=0, in_place=False):
    import bit_vq_routed_gb300 as bv
    g = ac.gen(seed + T * 31 + N * 7 + K)
    x, sx = _rows(g, T, K, pad)
    w, sw = _rows(g, N, K, pad, std=K ** -0.5)
    b = ac.normal(g, N, dtype=dt) if bias else None
    r = rc.wide(ac.normal(g, T, N, dtype=dt), pad) if residual else None
    y = r if in_place else rc.wide(torch.full((T, N), 3.0, dtype=dt, device="cuda"), pad)
    ws = torch.zeros(bv.moe_linear_8bit_workspace_size(T, N, K), dtype=torch.uint8, device="cuda")
    want, tol = rc.linear8_64(x, sx, w, sw, b, act, r, dt)
    bv.moe_linear_8bit(x, sx, w, sw, y, bias=b, act=act, residual=r, ws=ws)
    bv.moe_check_waits(ws)
    ac.within(y, want, tol, f"T={T} N={N} K={K}")
    return x, sx, w, sw, b, r, y


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("K", [16, 48, 128, 1040, 4096])
@pytest.mark.parametrize("T,N", [(1, 1), (1, 130), (3, 257), (8, 64), (9, 100), (16, 128), (17, 300), (33, 129), (64, 640),
                                 (65, 256), (130, 511), (257, 300)])
def test_sizes(dt, K, T, N):
    torch_cuda()
    _run(T, N, K, dt)


@pytest.mark.parametrize("T", [1, 8, 20, 100, 300])
@pytest.mark.parametrize("act", [0, 1, 2, 3, 4])
def test_epilogues(T, act):
    torch_cuda()
    for bias, residual in ((True, False), (True, True), (False, True)):
        _run(T, 203, 272, F16 if act % 2 else BF, act, bias, residual, pad=16)


@pytest.mark.parametrize("T,N,K", [(2, 4096, 4096), (5, 8200, 512), (8, 15000, 256), (48, 6144, 4096), (96, 6144, 2048), (700, 1100, 2064), (2048, 2304, 1024),
                                   (128, 512, 8192)])
def test_larger(T, N, K):
    torch_cuda()
    _run(T, N, K, bias=True, residual=True)


@pytest.mark.parametrize("T", [9, 15, 16, 17, 24, 31, 32])
@pytest.mark.parametrize("N,K", [(1, 16), (40, 1536), (2900, 1040), (4864, 512), (4865, 80), (7300, 528), (14593, 144),
                                 (2433, 5120), (64, 2560), (64, 2576)])
def test_9_to_32_tokens(T, N, K):
    """On both sides of each size at which another kernel takes them."""
    torch_cuda()
    _run(T, N, K, F16 if T % 2 else BF, T % 5, bias=True, residual=T % 3 == 0, pad=16)


@pytest.mark.parametrize("T,N,K", [(1, 2432, 2064), (8, 100, 6144), (8, 2433, 2560), (3, 4865, 2560), (2, 2500, 8192),
                                   (1, 17, 16384), (8, 700, 6160), (9, 40, 1536), (16, 2432, 1552), (16, 800, 6160),
                                   (11, 816, 8192), (13, 2433, 2576), (9, 4864, 7168), (17, 40, 2560), (32, 2432, 1040),
                                   (30, 8, 2576)])
def test_more_warps_for_more_inputs(T, N, K):
    torch_cuda()
    _run(T, N, K, BF if N % 2 else F16, 4, bias=True, residual=True, pad=32)


@pytest.mark.parametrize("T", [1, 30, 200])
def test_residual_in_place(T):
    torch_cuda()
    _run(T, 256, 256, residual=True, in_place=True)


@pytest.mark.parametrize("T", [1, 12, 90])
def test_columns_behind_y_and_what_is_not_finite(T):
    """What is not finite in one token or one output stays there; the columns
    behind a row of y are left alone."""
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    g = ac.gen(T)
    N, K = 150, 160
    x, sx = _rows(g, T, K)
    w, sw = _rows(g, N, K)
    sx[T // 2] = float("nan")
    sw[7] = float("inf")
    y = torch.full((T, N + 10), 9.0, dtype=BF, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    bv.moe_linear_8bit(x, sx, w, sw, y[:, :N], ws=ws)
    assert bool((y[:, N:] == 9).all())
    fine = torch.isfinite(y[:, :N])
    want = torch.ones(T, N, dtype=torch.bool, device="cuda")
    want[T // 2] = False
    want[:, 7] = False
    assert torch.equal(fine, want)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_same_bits_again_on_another_stream_and_in_a_graph(T):
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    x, sx, w, sw, b, r, y = _run(T, 384, 512, bias=True)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    y2 = torch.empty_like(y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bv.moe_linear_8bit(x, sx, w, sw, y2, bias=b, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(y, y2)
    y2.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bv.moe_linear_8bit(x, sx, w, sw, y2, bias=b, ws=ws)
    graph.replay()
    assert torch.equal(y, y2)
