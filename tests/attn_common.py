"""Shared pieces of the attention-side tests: plain 64-bit implementations
and the tolerances, derived from the operators' stated arithmetic.

Unit roundoffs: bf16 u = 2^-8, fp16 u = 2^-11, fp32 e = 2^-24.  Sums of n
fp32 terms, in any order and with any rounding of each partial sum (also by
truncation), are within n * 2^-23 * sum |terms|.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# half the distance of the smallest subnormals (results below the normal range)
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
E23 = 2.0 ** -23


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


# ------------------------------------------------------------------ linear

def act64(z, act):
    if act == 1:
        return torch.clamp(z, min=0)
    if act == 2:
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == 3:
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == 4:
        return z * torch.sigmoid(z)
    return z


def linear64(x, w, bias, act, residual):
    """(result, tolerance).  The pre-activation is off by at most
    (K + 1) 2^-23 (sum |x w| + |bias|); every activation here has a slope
    below 1.13; its own fp32 evaluation is within 16 e of (|z| + |act z|) (a
    few roundings, and functions good to a few units); then the residual's
    sum and the final rounding."""
    X, W = x.double(), w.double()
    z = X @ W.t()
    mag = X.abs() @ W.abs().t()
    if bias is not None:
        z = z + bias.double()
        mag = mag + bias.double().abs()
    a = act64(z, act)
    tol = 1.13 * (x.shape[1] + 1) * E23 * mag
    if act:
        tol = tol + 8 * E23 * (z.abs() + a.abs())
    y = a if residual is None else a + residual.double()
    u = U[x.dtype]
    tol = tol + E23 * y.abs()
    return y, (tol * (1 + u) + u * y.abs() + TINY[x.dtype])


# ------------------------------------------------------------------ attention

def attention64(q, kc, vc, cu_q, prefix_pages, prefix_len, page_table, seq_lens, scale):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits, sequence by
    sequence.  A score's sum of D products, its scaling and the subtraction
    of a reference move it by at most d = (D + 4) 2^-23 max(scale sum |q k|) + 2^-21,
    so a probability by a factor within e^(+-2d) (numerator and denominator: 2d
    each way); its rounding to the element type by u (an underflowing one by
    TINY against a largest of at least 2^-8); the sums by n 2^-23; the result's
    own rounding by u."""
    T, Hq, D = q.shape
    page, Hk = kc.shape[1], kc.shape[2]
    G = Hq // Hk
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    tlse = torch.zeros_like(lse)
    cu, lens = cu_q.tolist(), seq_lens.tolist()
    u, tiny = U[q.dtype], TINY[q.dtype]
    pp = prefix_pages.long()
    for b in range(len(lens)):
        t0, t1 = cu[b], cu[b + 1]
        n = t1 - t0
        if n == 0:
            continue
        m = min(max(lens[b], 0), page_table.shape[1] * page)
        own = page_table[b, :-(-m // page)].long()
        K = torch.cat((kc[pp].reshape(-1, Hk, D)[:prefix_len], kc[own].reshape(-1, Hk, D)[:m])).double()
        V = torch.cat((vc[pp].reshape(-1, Hk, D)[:prefix_len], vc[own].reshape(-1, Hk, D)[:m])).double()
        K, V = K.repeat_interleave(G, 1).transpose(0, 1), V.repeat_interleave(G, 1).transpose(0, 1)
        Q = q[t0:t1].double().transpose(0, 1)
        S = scale * (Q @ K.transpose(1, 2))
        i = torch.arange(n, device=q.device)[:, None]
        j = torch.arange(K.shape[1], device=q.device)[None]
        seen = (j < prefix_len) | (j - prefix_len <= m - n + i)
        S = S.masked_fill(~seen, -math.inf)
        if K.shape[1] == 0:
            continue
        some = seen.any(1)
        P = torch.where(some[:, None], torch.softmax(S, -1), torch.zeros_like(S))
        mag = (scale * (Q.abs() @ K.abs().transpose(1, 2))).masked_fill(~seen, 0.0)
        d = (D + 4) * E23 * mag.amax(-1, keepdim=True) + 2.0 ** -21
        N = K.shape[1] + 8
        A = P @ V.abs()
        o = P @ V
        vmax = V.abs().amax((1, 2))[:, None, None]
        out[t0:t1] = o.transpose(0, 1)
        tol[t0:t1] = ((u + torch.expm1(4 * d) + 4 * N * E23) * (1 + u) * A + u * o.abs() + N * tiny * 2.0 ** 8 * vmax
                      + tiny).transpose(0, 1)
        lse[t0:t1] = torch.logsumexp(S, -1).t()  # (of no key at all: -infinity)
        tlse[t0:t1] = (d[..., 0] + 2 * N * E23 + 4 * E23 * lse[t0:t1].t().abs()).t()
    return out, lse, tol, tlse


def within(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - want).abs() > tol
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst by " \
        f"{float(((got - want).abs() / tol.clamp_min(1e-300)).max()):.2f} times the tolerance, first at " \
        f"{torch.nonzero(bad)[0].tolist()}"
