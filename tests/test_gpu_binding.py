"""The short way from Python to the norm, the 8-bit rows and products and the choice
by score: the same results as by way of ctypes, and the same refusals."""
import pytest

torch = pytest.importorskip("torch")
import attn_common as ac  # noqa: E402
import rows_common as rc  # noqa: E402
from gpu_common import torch_cuda  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F32, E4M3 = torch.bfloat16, torch.float32, rc.E4M3
QUICK = ("_quick_norm", "_quick_rows", "_quick_linear_8bit", "_quick_route_scored")


@pytest.fixture(params=[True, False])
def ways(request, monkeypatch):
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    bv.load()
    assert all(getattr(bv, n) is not bv._look_again for n in QUICK)  # (built and loaded)
    if not request.param:
        for n in QUICK:
            monkeypatch.setattr(bv, n, bv._look_again)
    return bv


def _calls(bv, stream=None):
    """One call of each, and what they wrote."""
    g = ac.gen(1)
    T, H, N, E, k = 5, 160, 70, 64, 6
    x, res, w = ac.normal(g, T, H, dtype=F32), ac.normal(g, T, H), ac.normal(g, H)
    h, y = torch.empty_like(res), torch.empty_like(res)
    q, s = torch.zeros(T, H, dtype=E4M3, device="cuda"), torch.zeros(T, device="cuda")
    wq, ws = torch.zeros(N, H, dtype=E4M3, device="cuda"), torch.zeros(N, device="cuda")
    out, bias = torch.zeros(T, N, dtype=BF, device="cuda"), ac.normal(g, N)
    room = torch.zeros(256, dtype=torch.uint8, device="cuda")
    logits, rb = ac.normal(g, T, E, dtype=F32), ac.normal(g, E, dtype=F32, std=0.1)
    ids, weights = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    w32 = ac.normal(g, N, H, dtype=F32)
    torch.cuda.synchronize()
    bv.moe_rms_norm(x, w, 1e-6, residual=res, h=h, y=y, q=q, scales=s, stream=stream)
    bv.moe_quantize_rows(w32, wq, ws, stream)
    bv.moe_linear_8bit(q, s, wq, ws, out, bias=bias, act=bv.MOE_ACT_SILU, residual=y[:, :N], ws=room, stream=stream)
    bv.moe_route_scored(logits, k, ids, weights, scoring=1, bias=rb, groups=8, top_groups=3, group_top=2, renormalize=True,
                        scale=2, stream=stream)
    torch.cuda.synchronize()
    return [t.clone() for t in (h, y, q.view(torch.uint8), s, wq.view(torch.uint8), ws, out, ids, weights)]


def test_both_ways_and_every_stream_give_the_same(ways, monkeypatch):
    got = _calls(ways)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        assert all(torch.equal(a, b) for a, b in zip(got, _calls(ways, stream)))
    with torch.cuda.stream(side):
        assert all(torch.equal(a, b) for a, b in zip(got, _calls(ways)))
    for n in QUICK:
        monkeypatch.setattr(ways, n, ways._look_again)
    assert all(torch.equal(a, b) for a, b in zip(got, _calls(ways)))


def test_both_ways_refuse_the_same(ways):
    bv = ways
    z = lambda *s, dtype=BF, device="cuda": torch.zeros(*s, dtype=dtype, device=device)  # noqa: E731
    x, y, q, s = z(2, 64), z(2, 64), z(2, 64, dtype=E4M3), z(2, dtype=F32)
    wq, ws, o, room = z(32, 64, dtype=E4M3), z(32, dtype=F32), z(2, 32), z(256, dtype=torch.uint8)
    lg, ids, wt = z(2, 16, dtype=F32), z(2, 4, dtype=torch.int32), z(2, 4, dtype=F32)
    n = bv.moe_launch_count()
    norm = lambda **k: bv.moe_rms_norm(**dict(dict(x=x, weight=z(64), eps=1e-6, y=y), **k))  # noqa: E731
    lin = lambda **k: bv.moe_linear_8bit(**dict(dict(x=q, x_scales=s, w=wq, w_scales=ws, y=o, ws=room), **k))  # noqa: E731
    route = lambda **k: bv.moe_route_scored(**dict(dict(logits=lg, k=4, ids=ids, weights=wt), **k))  # noqa: E731
    for call, kw in ((norm, dict(x=z(2, 64, dtype=torch.float16))), (norm, dict(x=z(2, 64, device="cpu"))),
                     (norm, dict(x=z(64, 2).t())), (norm, dict(weight=z(63))), (norm, dict(weight=z(64, dtype=F32))),
                     (norm, dict(residual=z(3, 64))), (norm, dict(y=z(2, 65))), (norm, dict(y=y.float())),
                     (norm, dict(residual=x, h=z(2, 64, device="cpu"))), (norm, dict(q=y, scales=s)),
                     (norm, dict(q=q, scales=z(3, dtype=F32))), (norm, dict(q=q, scales=z(2))),
                     (lambda **k: bv.moe_quantize_rows(**k), dict(x=x, q=y, scales=s)),
                     (lambda **k: bv.moe_quantize_rows(**k), dict(x=x, q=z(3, 64, dtype=E4M3), scales=s)),
                     (lambda **k: bv.moe_quantize_rows(**k), dict(x=z(2, 64, dtype=torch.int16), q=q, scales=s)),
                     (lambda **k: bv.moe_quantize_rows(**k), dict(x=x, q=q, scales=z(2, device="cpu", dtype=F32))),
                     (lin, dict(x=x)), (lin, dict(w=z(32, 48, dtype=E4M3))), (lin, dict(x_scales=z(3, dtype=F32))),
                     (lin, dict(w_scales=z(64, dtype=F32)[::2])), (lin, dict(y=z(2, 33))), (lin, dict(y=z(2, 32, dtype=F32))),
                     (lin, dict(bias=z(32, dtype=torch.float16))), (lin, dict(residual=z(2, 31))),
                     (lin, dict(ws=room.cpu())), (lin, dict(w=wq.cpu())), (route, dict(logits=z(2, 16))),
                     (route, dict(logits=z(2, 32, dtype=F32)[:, ::2])), (route, dict(ids=z(2, 4, dtype=torch.int64))),
                     (route, dict(weights=z(2, 5, dtype=F32))), (route, dict(bias=z(15, dtype=F32))), (route, dict(k=5))):
        with pytest.raises(ValueError):
            call(**kw)
    for call, kw, status in ((norm, dict(eps=-1.0), bv.MOE_ERR_INVALID_ARG), (norm, dict(y=None), bv.MOE_ERR_INVALID_ARG),
                             (norm, dict(q=q), bv.MOE_ERR_INVALID_ARG), (norm, dict(h=y), bv.MOE_ERR_INVALID_ARG),
                             (lin, dict(ws=None), bv.MOE_ERR_WORKSPACE), (lin, dict(ws=room[:8]), bv.MOE_ERR_WORKSPACE),
                             (lin, dict(act=9), bv.MOE_ERR_INVALID_ARG), (route, dict(groups=3), bv.MOE_ERR_INVALID_ARG),
                             (route, dict(scoring=7), bv.MOE_ERR_INVALID_ARG), (route, dict(scale=float("nan")), bv.MOE_ERR_INVALID_ARG)):
        with pytest.raises(bv.MoeError) as e:
            call(**kw)
        assert e.value.status == status
    assert bv.moe_launch_count() == n


def test_unusual_but_allowed(ways):
    """Rows one element long, a single strided row, no tensors but x to tell the type."""
    bv = ways
    x = torch.randn(4, 1, device="cuda")
    y = torch.zeros(4, 1, dtype=BF, device="cuda")
    bv.moe_rms_norm(x, None, 0.0, y=y)
    assert torch.equal(y, torch.sign(x).to(BF))
    col = torch.randn(64, 1, dtype=BF, device="cuda").t()  # [1, 64], strides (1, 1)
    q, s = torch.zeros(1, 64, dtype=E4M3, device="cuda"), torch.zeros(1, device="cuda")
    bv.moe_rms_norm(col, None, 1e-6, q=q, scales=s)
    y64, rel = rc.rms64(col, None, 1e-6)
    rc.check_rows8(q, s, y64, rel, "one row")
    bv.moe_quantize_rows(col, q, s)
    assert torch.equal(q.double(), rc.eighths(rc.rows8_64(col)[0]))
