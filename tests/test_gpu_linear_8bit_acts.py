"""The activations of the 8-bit products, point by point: with inputs of zeros the
pre-activation is the bias, which 16 bits hold exactly."""
import pytest

torch = pytest.importorskip("torch")
import attn_common as ac  # noqa: E402
import rows_common as rc  # noqa: E402
from gpu_common import torch_cuda  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16


def _points(dt):
    """Every 16-bit value between 2^-14 and 16 of both signs, zeros, large ones."""
    bits = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16)
    v = bits.view(dt)
    a = v.float().abs()
    v = v[(a >= 2.0 ** -14) & (a <= 16.0)]
    return torch.cat((v, torch.tensor([0.0, -0.0, 40.0, -40.0, 300.0, -300.0, 6e4, -6e4, 1e-6, -1e-6]).to(dt))).cuda()


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("act", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("T", [1, 24, 40, 300])
@pytest.mark.parametrize("residual", [False, True])
def test_points(dt, act, T, residual):
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    z = _points(dt)
    N, K = z.shape[0], 128
    x, w = (torch.zeros(n, K, device="cuda").to(rc.E4M3) for n in (T, N))
    sx, sw = torch.ones(T, device="cuda"), torch.ones(N, device="cuda")
    r = ac.normal(ac.gen(T), T, N, dtype=dt, std=1e-3) if residual else None
    y = torch.full((T, N), 3.0, dtype=dt, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    bv.moe_linear_8bit(x, sx, w, sw, y, bias=z, act=act, residual=r, ws=ws)
    bv.moe_check_waits(ws)
    a = ac.act64(z.double(), act)
    if act == 2:  # (1 + erf cancels in 64 bits too)
        a = 0.5 * z.double() * torch.special.erfc(-z.double() / 2 ** 0.5)
    if act == 3:
        a = z.double() * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z.double() + 0.044715 * z.double() ** 3))
    want = a[None, :] + (r.double() if residual else 0.0)
    # the activation is off by 2^-16 of itself (what fp32 flushes to zero: 2^-120), the sum by
    # 2^-24 of its result, the result by half a step
    tol = a.abs()[None, :] * 2.0 ** -16 + 2.0 ** -120 + want.abs() * 2.0 ** -24
    ac.within(y, want.expand(T, N), tol * (1 + ac.U[dt]) + ac.U[dt] * want.abs() + ac.TINY[dt], f"act {act}")


@pytest.mark.parametrize("T", [1, 24, 40, 300])
@pytest.mark.parametrize("act", [0, 1, 2, 3, 4])
def test_infinity_and_nan(T, act):
    torch_cuda()
    import bit_vq_routed_gb300 as bv
    z = torch.tensor([float("inf"), float("nan"), 1.0] * 16, dtype=BF, device="cuda")
    N, K = z.shape[0], 64
    x, w = (torch.zeros(n, K, device="cuda").to(rc.E4M3) for n in (T, N))
    y = torch.zeros(T, N, dtype=BF, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    bv.moe_linear_8bit(x, torch.ones(T, device="cuda"), w, torch.ones(N, device="cuda"), y, bias=z, act=act, ws=ws)
    assert bool((y[:, 0::3] == float("inf")).all()) and bool(torch.isnan(y[:, 1::3]).all())
    assert bool(torch.isfinite(y[:, 2::3]).all())
