"""Shared pieces of the tests of the norm, the 8-bit rows and products and the
choice of experts by score: plain 64-bit implementations and the tolerances,
derived from the operators' stated arithmetic.

e4m3: 3 fraction bits, smallest normal 2^-6, so a rounding is off by at most
2^-4 of the value, or by 2^-10 below the normal range.
"""
import math

import torch

import attn_common as ac

E4M3 = torch.float8_e4m3fn
LEAST = 1e-30
E24 = 2.0 ** -24


def eighths(v):
    """Nearest e4m3 value (halves to even) of |v| <= 448, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def wide(t, pad):
    """t as the leading columns of longer rows (pad more elements)."""
    if not pad:
        return t
    w = torch.full((t.shape[0], t.shape[1] + pad), 7, dtype=torch.float32, device=t.device).to(t.dtype)
    w[:, :t.shape[1]] = t
    return w[:, :t.shape[1]]


def rms64(h, weight, eps):
    """(y, its relative error in fp32): 16 squares a thread and 10 rounds of
    sums, the division and eps make 28 roundings of the mean, half of that after
    the root; the root is good to 4 units and two products follow: 20 units."""
    h = h.double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return (y if weight is None else y * weight.double()), 20 * E24


def rows8_64(v):
    """(v * 448 / a, a) in 64 bits."""
    a = v.double().abs().amax(1, keepdim=True).clamp_min(LEAST)
    return v.double() * 448 / a, a[:, 0]


def check_rows8(q, scales, v, rel, what):
    """8-bit rows of a v that fp32 knows up to a relative error rel: the largest
    magnitude and the quotient add 4 roundings and v's own error twice."""
    want, a = rows8_64(v)
    d = 2 * rel + 4 * E24
    ac.within(scales, a / 448, a / 448 * d, what + " scales")
    ac.within(q, want, want.abs() * (2.0 ** -4 + 2 * d) + 2.0 ** -10, what + " q")


def linear8_64(x, sx, w, sw, bias, act, residual, dtype):
    """attn_common.linear64 for 8-bit rows: the products are exact, the scales
    add two roundings to the sum."""
    X, W = x.double() * sx.double()[:, None], w.double() * sw.double()[:, None]
    z, mag = X @ W.t(), X.abs() @ W.abs().t()
    if bias is not None:
        z = z + bias.double()
        mag = mag + bias.double().abs()
    a = ac.act64(z, act)
    tol = 1.13 * (x.shape[1] + 3) * ac.E23 * mag
    if act:
        tol = tol + 8 * ac.E23 * (z.abs() + a.abs())
    y = a if residual is None else a + residual.double()
    u = ac.U[dtype]
    tol = tol + ac.E23 * y.abs()
    return y, tol * (1 + u) + u * y.abs() + ac.TINY[dtype]


def scored64(logits, k, sigmoid, bias, groups, top_groups, group_top, renorm, scale):
    """(ids, weights) on the CPU in 64 bits, token by token."""
    v = logits.double().cpu()
    T, E = v.shape
    n = E // groups
    score = torch.sigmoid(v) if sigmoid else torch.softmax(v, -1)
    choice = score if bias is None else score + bias.double().cpu()
    if bias is None and not (groups > 1 and group_top == 2):
        choice = v  # (the scores' order, also where 64 bits round them to one value)
    ids = []
    for row in choice.tolist():
        best = [sum(sorted(row[g * n:(g + 1) * n], reverse=True)[:group_top]) for g in range(groups)]
        kept = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
        left = sorted(e for g in kept for e in range(g * n, (g + 1) * n))
        ids.append(sorted(left, key=lambda e: (-row[e], e))[:k])
    ids = torch.tensor(ids).view(T, k)
    w = torch.gather(score, 1, ids)
    if renorm:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return ids.to(torch.int32), w * scale
