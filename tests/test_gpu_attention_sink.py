"""moe_prefix_attention where nearly all of a row's weight is on one key of
small value (an attention sink) and its result comes from thousands of keys far
below the maximum, and where scores are so large that their product with
log2(e) is coarsely rounded."""
import math

import pytest

from gpu_common import torch_cuda

pytestmark = pytest.mark.gpu


def _call(q, K, V, scale):
    """out and lse of q [T, Hq, D] over K, V [N, Hk, D] as a prefix that every
    token sees (one sequence that holds nothing of its own)."""
    torch = torch_cuda()
    import bit_vq_routed_gb300 as bv
    T, Hq, D = q.shape
    N, Hk = K.shape[:2]
    kc, vc = K.view(N // 128, 128, Hk, D), V.view(N // 128, 128, Hk, D)
    i32 = dict(dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(T, Hq, device="cuda")
    ws = torch.zeros(bv.moe_prefix_attention_workspace_size(T, Hq, Hk, D), dtype=torch.uint8, device="cuda")
    bv.moe_prefix_attention(q, kc, vc, torch.tensor([0, T], **i32), torch.arange(N // 128, **i32), N,
                            torch.zeros(1, 1, **i32), torch.zeros(1, **i32), scale, out, lse, ws)
    assert int(ws[8:12].view(torch.int32).item()) == 0
    return out, lse


# The tolerance (N keys, u the element type's unit roundoff, E = 2^-23):
#   - a score's sum of D products, its scaling, and the subtraction of the reference move it by at most
#     d = (D + 4) E max(scale sum |q k|) + 2^-21, so a probability and the sum by e^(+-2d) each way;
#   - the probability's rounding to the element type by u, the sums by N E, the result's rounding by u;
#   - what is below the type's normal range is rounded to half its smallest subnormal, TINY = 2^-25 in fp16.
#     The row's own largest probability is at least 2^7 there (the reference is never above the row's maximum,
#     and the kernel's probabilities are relative to it times 2^7), so each key adds at most 2^-32 |v|.
def _want(torch, ac, q, K, V, scale, h, shift):
    """Out, lse and their tolerances for key head h, in 64 bits."""
    dt, D, N = q.dtype, q.shape[2], K.shape[0]
    G = q.shape[1] // K.shape[1]
    Q, k, v = q[:, h * G:(h + 1) * G].reshape(-1, D).double(), K[:, h].double(), V[:, h].double()
    S = scale * (Q @ k.t())
    d = (D + 4) * ac.E23 * (scale * (Q.abs() @ k.abs().t())).amax(1, keepdim=True) + 2.0 ** -21
    P = torch.softmax(S, 1)
    o, A, u = P @ v, P @ v.abs(), ac.U[dt]
    tol = (u + torch.expm1(4 * d) + 4 * N * ac.E23) * (1 + u) * A + u * o.abs()
    tol = tol + N * ac.TINY[dt] * 2.0 ** -shift * float(v.abs().max()) + ac.TINY[dt]
    l = torch.logsumexp(S, 1)
    return o, l, tol, d[:, 0] + 2 * N * ac.E23 + 4 * ac.E23 * l.abs()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("gap", [10, 14, 16, 17, 18, 20])
@pytest.mark.parametrize("T,heads,group,N", [(1024, 4, 8, 8192), (600, 2, 1, 2048), (3, 1, 4, 16384), (1, 64, 1, 8192)])
def test_sink(T, heads, group, N, gap, dtype):
    # scores of the sink: gap; of all others: 0.  Values of the sink: 0; of the others: about 1, of one sign.
    torch = torch_cuda()
    import attn_common as ac
    dt, D = getattr(torch, dtype), 64
    g = ac.gen(gap)
    q = torch.zeros(T, heads * group, D, dtype=dt, device="cuda")
    q[..., 0] = 4.0
    q[..., 1:] = ac.normal(g, T, heads * group, D - 1, dtype=dt)
    K = torch.zeros(N, heads, D, dtype=dt, device="cuda")
    K[0, :, 0] = gap * 2.0  # (times 4, times the scale 1/8)
    V = ac.normal(g, N, heads, D, dtype=dt, std=0.1) + 1
    V[0] = 0
    out, lse = _call(q, K, V, 0.125)
    G = group
    for h in range(heads):
        o, l, to, tl = _want(torch, ac, q, K, V, 0.125, h, 7)
        ac.within(out[:, h * G:(h + 1) * G].reshape(-1, D), o, to, f"out, head {h}")
        ac.within(lse[:, h * G:(h + 1) * G].reshape(-1), l, tl, f"lse, head {h}")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("size", [2.0 ** 9, 2.0 ** 11, 2.0 ** 13])
@pytest.mark.parametrize("T", [1, 300])
def test_probabilities_of_large_scores_stay_in_range(T, size, dtype):
    # Scores up to 2^27, where the maximum times log2(e) is rounded by up to 2^3, and values that are the same for
    # all keys: the result is that value, whatever the keys' weights are, as long as their numerator and
    # denominator stay in range (the result's rounding and the probabilities': 2 u, the sums N E each).
    torch = torch_cuda()
    import attn_common as ac
    dt, D, N = getattr(torch, dtype), 64, 1024
    q = torch.full((T, 4, D), size, dtype=dt, device="cuda")
    K = torch.full((N, 1, D), size / 4, dtype=dt, device="cuda")
    V = (ac.normal(ac.gen(5), 1, 1, D, dtype=dt) + 3).expand(N, 1, D).contiguous()
    for scale in (0.125, 0.1171875, 0.1328125):
        out, _ = _call(q, K, V, scale)
        o = V[0, 0].double().expand(T, 4, D)
        ac.within(out, o, (2 * ac.U[dt] + 4 * N * ac.E23) * o.abs(), f"scale {scale}")
