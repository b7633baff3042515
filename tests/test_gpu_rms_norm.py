"""moe_rms_norm and moe_quantize_rows against 64 bits."""
import pytest

torch = pytest.importorskip("torch")
import attn_common as ac  # noqa: E402
import rows_common as rc  # noqa: E402
from gpu_common import torch_cuda  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _call(x, dt, res, weight, eps=1e-6, y=True, q=True, pad=0, in_place=False, stream=None):
    import bit_vq_routed_gb300 as bv
    T, H = x.shape
    empty = lambda t: rc.wide(torch.full((T, H), 3.0, device="cuda").to(t), pad)  # noqa: E731
    h = None if res is None else res if in_place else empty(dt)
    yo, qo = empty(dt) if y else None, empty(rc.E4M3) if q else None
    sc = torch.full((T,), 5.0, device="cuda") if q else None
    bv.moe_rms_norm(x, weight, eps, residual=res, h=h, y=yo, q=qo, scales=sc, dtype=dt, stream=stream)
    return h, yo, qo, sc


def _check(x, dt, res, weight, got, eps=1e-6):
    h, y, q, sc = got
    v = x.double()
    if res is not None:
        want = (x.float() + res.float()).to(dt)
        assert torch.equal(h, want)
        v = want.double()
    y64, rel = rc.rms64(v, weight, eps)
    if y is not None:
        u = ac.U[dt]
        ac.within(y, y64, y64.abs() * (rel * (1 + u) + u) + ac.TINY[dt], "y")
    if q is not None:
        rc.check_rows8(q, sc, y64, rel, "rows")


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("x32", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H,pad", [(1, 1, 0), (3, 7, 0), (5, 8, 0), (2, 31, 1), (7, 64, 8), (1, 4096, 0), (700, 256, 0),
                                     (33, 2051, 24), (9, 4104, 24), (2, 16384, 0), (3, 16383, 5), (1300, 520, 0)])
def test_norm(dt, x32, residual, T, H, pad):
    torch_cuda()
    g = ac.gen(T * H + x32)
    x = rc.wide(ac.normal(g, T, H, dtype=F32 if x32 else dt), pad)
    res = rc.wide(ac.normal(g, T, H, dtype=dt, std=2.0), pad) if residual else None
    weight = ac.normal(g, H, dtype=dt)
    _check(x, dt, res, weight, _call(x, dt, res, weight, pad=pad))


@pytest.mark.parametrize("y,q", [(True, False), (False, True)])
def test_one_output_and_no_weight(y, q):
    torch_cuda()
    g = ac.gen(1)
    x, res = ac.normal(g, 40, 1000, dtype=F32), ac.normal(g, 40, 1000)
    _check(x, BF, res, None, _call(x, BF, res, None, y=y, q=q))


def test_h_in_the_residuals_place():
    torch_cuda()
    g = ac.gen(2)
    for H in (1024, 1023):
        x, res = ac.normal(g, 2000, H, dtype=F32), ac.normal(g, 2000, H)
        weight, old = ac.normal(g, H), res.clone()
        got = _call(x, BF, res, weight, in_place=True)
        assert got[0] is res
        _check(x, BF, old, weight, got)
        # and the norm of the stored sum is the same as that of a call on it
        again = _call(res, BF, None, weight)
        assert torch.equal(again[1], got[1]) and torch.equal(again[2].view(torch.uint8), got[2].view(torch.uint8))
        assert torch.equal(again[3], got[3])


def test_no_h_wanted_and_columns_behind_the_rows():
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    g = ac.gen(3)
    for H in (128, 125):
        x, res, weight = ac.normal(g, 6, H), ac.normal(g, 6, H), ac.normal(g, H)
        y = torch.full((6, H + 16), 9.0, dtype=BF, device="cuda")
        q = torch.full((6, H + 16), 9.0, device="cuda").to(rc.E4M3)
        sc = torch.empty(6, device="cuda")
        bv.moe_rms_norm(x, weight, 1e-6, residual=res, y=y[:, :H], q=q[:, :H], scales=sc)
        assert bool((y[:, H:] == 9).all()) and bool((q[:, H:].float() == 9).all())
        y64, rel = rc.rms64((x.float() + res.float()).to(BF), weight, 1e-6)
        ac.within(y[:, :H], y64, y64.abs() * (rel + 2.0 ** -8) + ac.TINY[BF], "y")
        rc.check_rows8(q[:, :H], sc, y64, rel, "rows")


def test_rows_of_zeros_and_rows_that_are_not_finite():
    torch_cuda()
    x = ac.normal(ac.gen(4), 5, 96, dtype=F32)
    x[1] = 0
    x[2, 40] = float("nan")
    x[3, 7] = float("inf")
    h, y, q, sc = _call(x, BF, None, None)
    back = q.float() * sc[:, None]
    assert bool((y[1] == 0).all()) and bool((back[1] == 0).all()) and bool(torch.isfinite(sc[1]))
    for t in (0, 4):
        assert bool(torch.isfinite(y[t]).all()) and bool(torch.isfinite(back[t]).all())
    assert bool(torch.isnan(y[2]).all()) and not bool(torch.isfinite(y[3]).all())
    assert not bool(torch.isfinite(sc[2])) and not bool(torch.isfinite(sc[3]))
    _check(x[4:], BF, None, None, (None, y[4:], q[4:], sc[4:]))


def test_eps_and_small_rows():
    torch_cuda()
    x = ac.normal(ac.gen(5), 4, 512, dtype=F32, std=1e-4)
    for eps in (0.0, 1e-6, 0.5):
        _check(x, F16, None, None, _call(x, F16, None, None, eps=eps), eps=eps)


def test_stream_and_graph():
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    g = ac.gen(6)
    x, res, weight = ac.normal(g, 64, 768, dtype=F32), ac.normal(g, 64, 768), ac.normal(g, 768)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _call(x, BF, res, weight, stream=side)
    side.synchronize()
    _check(x, BF, res, weight, got)
    h, y = torch.empty_like(res), torch.empty_like(res)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bv.moe_rms_norm(x, weight, 1e-6, residual=res, h=h, y=y)
        bv.moe_rms_norm(y, weight, 1e-6, residual=h, h=h, y=y)
    res.copy_(ac.normal(g, 64, 768))
    graph.replay()
    h1 = (x.float() + res.float()).to(BF)
    y1 = torch.empty_like(h1)
    bv.moe_rms_norm(h1, weight, 1e-6, y=y1)
    assert torch.equal(h, (y1.float() + h1.float()).to(BF))


# ------------------------------------------------------------------ rows to 8 bits

@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("T,H,pad", [(1, 1, 0), (5, 16, 0), (3, 33, 2), (64, 4096, 0), (40, 1000, 8), (2, 16384, 0), (900, 200, 0),
                                     (3, 16385, 0), (700, 20000, 8), (2, 50001, 7)])
def test_rows_of_16_bits_are_rounded_exactly(dt, T, H, pad):
    """448 x / a is a quotient of two short numbers: it is a halfway value or
    further from one than fp32 can miss, so every value rounds as in 64 bits."""
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    g = ac.gen(T + H)
    x = ac.normal(g, T, H, dtype=dt)
    x[0, 0] = 7.0 if dt == BF else 3.5  # (quotients x * 64, x * 128: halfway values among them)
    x[0, 1:] = x[0, 1:].clamp(-3.5, 3.5)
    x = rc.wide(x, pad)
    q = rc.wide(torch.zeros(T, H, device="cuda").to(rc.E4M3), pad)
    sc = torch.empty(T, device="cuda")
    bv.moe_quantize_rows(x, q, sc)
    want, a = rc.rows8_64(x)
    assert torch.equal(q.double(), rc.eighths(want))
    ac.within(sc, a / 448, a / 448 * 2.0 ** -24, "scales")


def test_rows_of_32_bits():
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    g = ac.gen(9)
    x = ac.normal(g, 300, 1000, dtype=F32) * torch.exp(4 * ac.normal(g, 300, 1, dtype=F32))
    x[0], x[1] = 0, x[1] * 1e30
    x[2] = x[2].abs().clamp(0.5, 3) * 1e38
    x[3] *= 1e-36
    q, sc = torch.empty(300, 1000, dtype=rc.E4M3, device="cuda"), torch.empty(300, device="cuda")
    bv.moe_quantize_rows(x, q, sc)
    rc.check_rows8(q, sc, x, 0.0, "rows")
    x[5, 999], x[6, 0] = float("nan"), float("-inf")
    bv.moe_quantize_rows(x, q, sc)
    assert torch.isfinite(sc).tolist() == [t not in (5, 6) for t in range(300)]
    # rows too long for registers
    x = ac.normal(g, 9, 30000, dtype=F32)
    x[3] = 0
    q, sc = torch.empty(9, 30000, dtype=rc.E4M3, device="cuda"), torch.empty(9, device="cuda")
    bv.moe_quantize_rows(x, q, sc)
    rc.check_rows8(q, sc, x, 0.0, "long rows")
    x[5, 29999], x[6, 0] = float("nan"), float("-inf")
    bv.moe_quantize_rows(x, q, sc)
    assert torch.isfinite(sc).tolist() == [t not in (5, 6) for t in range(9)]


def test_no_rows():
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    n = bv.moe_launch_count()
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    bv.moe_rms_norm(z(0, 64), z(64), 1e-6, y=z(0, 64))
    bv.moe_quantize_rows(z(0, 64), z(0, 64, dtype=rc.E4M3), z(0, dtype=F32))
    assert bv.moe_launch_count() == n


@pytest.mark.parametrize("H", [64, 1000, 2048, 4096, 4944, 6144, 8192, 9000, 333])
def test_a_row_alone_and_among_many(H):
    """Bit for bit the same, whatever the number of rows, the outputs and the type
    of x make of the launch."""
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    g = ac.gen(H)
    T = 900
    x, weight = ac.normal(g, T, H), ac.normal(g, H)
    zero = torch.zeros(T, H, dtype=BF, device="cuda")
    _, y, q, sc = _call(x, BF, None, weight)
    for rows in (slice(0, 1), slice(5, 6), slice(100, 300)):
        for kw in (dict(), dict(q=False), dict(y=False)):
            got = _call(x[rows], BF, None, weight, **kw)
            assert got[1] is None or torch.equal(got[1], y[rows])
            assert got[2] is None or (torch.equal(got[2].view(torch.uint8), q[rows].view(torch.uint8)) and torch.equal(got[3], sc[rows]))
    for other in (x, x.float()):
        got = _call(other, BF, zero, weight)
        assert torch.equal(got[1], y) and torch.equal(got[3], sc) and torch.equal(got[2].view(torch.uint8), q.view(torch.uint8))
