"""moe_rms_norm's 8-bit rows: rows of zeros and rows whose norm lies below the
least magnitude, at every eps; and each value the nearest of the formula's, in which
a row's root cancels out:  y 448 / max |y| = h w 448 / max |h w|."""
import pytest

torch = pytest.importorskip("torch")
import attn_common as ac  # noqa: E402
import rows_common as rc  # noqa: E402
from gpu_common import torch_cuda  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _norm(x, weight, eps, dt, residual=None):
    import bit_vq_routed_gb300 as bv
    T, H = x.shape
    y, q = torch.full((T, H), 3.0, dtype=dt, device="cuda"), torch.full((T, H), 3.0, device="cuda").to(rc.E4M3)
    sc = torch.full((T,), 5.0, device="cuda")
    bv.moe_rms_norm(x, weight, eps, residual=residual, y=y, q=q, scales=sc, dtype=dt)
    return y, q, sc


# (sizes of whole pieces and of single elements, 8 and 16 of them a thread)
SIZES = [1, 64, 63, 4096, 4095, 9000, 9001]


@pytest.mark.parametrize("H", SIZES)
@pytest.mark.parametrize("eps", [1e-6, 1e-12, 1e-20, 1e-38])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_of_zeros(H, eps, residual):
    torch_cuda()
    g = ac.gen(H)
    x = ac.normal(g, 5, H, dtype=F32)
    x[1], x[3] = 0, -0.0
    res = torch.zeros(5, H, dtype=BF, device="cuda") if residual else None
    y, q, sc = _norm(x, ac.normal(g, H), eps, BF, res)
    for t in (1, 3):
        assert bool((y[t] == 0).all()) and bool((q[t].float() == 0).all())
        ac.within(sc[t], torch.tensor(rc.LEAST / 448, device="cuda", dtype=torch.float64), rc.LEAST / 448 * 2.0 ** -22, "scale")
    assert bool(torch.isfinite(q.float()).all()) and bool(torch.isfinite(sc).all())


@pytest.mark.parametrize("H", SIZES)
@pytest.mark.parametrize("eps", [1e-6, 1e-12, 1e-13])
def test_rows_below_the_least_magnitude(H, eps):
    """|y| = |x| / sqrt(eps) at most 1e-31 to 1e-30: counted against 1e-30, so small
    quotients (1e-13: r = 3e6, 448 r / 1e-30 past fp32)."""
    torch_cuda()
    g = ac.gen(H + 1)
    top = eps ** 0.5 * 1e-30
    x = (torch.rand(4, H, generator=g, device="cuda") - 0.5) * 2 * top
    x[2] *= 0.1
    x[3] = 0
    x[3, 0] = 0.9 * top
    for weight in (None, (1 + torch.rand(H, generator=g, device="cuda")).to(BF) / 2):
        y, q, sc = _norm(x, weight, eps, BF)
        y64, rel = rc.rms64(x, weight, eps)
        # (h w below fp32's normal range: off by 2^-150, times r 448 / 1e-30)
        want, a = rc.rows8_64(y64)
        low = 2.0 ** -149 * eps ** -0.5 * 448 / rc.LEAST
        d = 2 * rel + 4 * rc.E24
        ac.within(sc, a / 448, a / 448 * d, "scales")
        ac.within(q, want, want.abs() * (2.0 ** -4 + 2 * d) + 2.0 ** -10 + low, "q")


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("T,H", [(3, 64), (200, 4096), (90, 4097), (30, 9000), (1300, 520)])
@pytest.mark.parametrize("residual", [False, True])
def test_values_are_the_nearest(dt, T, H, residual):
    """bf16: h w has 16 bits, so its quotient is a halfway value of e4m3 or further
    than 2^-22 from one, and fp32's correctly rounded quotient falls as the exact one
    does.  fp16: 22 bits; the quotient is known to 2^-22 of itself."""
    torch_cuda()
    g = ac.gen(T + H)
    x = ac.normal(g, T, H, dtype=F32 if residual else dt, std=2.0)
    res = ac.normal(g, T, H, dtype=dt) if residual else None
    weight = ac.normal(g, H, dtype=dt)
    _, q, sc = _norm(x, weight, 1e-6, dt, res)
    h = x.double() if res is None else (x + res.float()).to(dt).double()
    v = h * weight.double()
    want = v * 448 / v.abs().amax(1, keepdim=True)
    got = q.double()
    if dt == BF:
        assert torch.equal(got, rc.eighths(want))
    else:
        near = (got == rc.eighths(want)) | (got == rc.eighths(want * (1 - 2.0 ** -22))) | \
            (got == rc.eighths((want * (1 + 2.0 ** -22)).clamp(-448, 448)))
        assert bool(near.all())
