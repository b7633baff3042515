r"""The attention side of a decoder layer, over a paged cache whose sequences
share a prefix, and the layer as a whole with the routed experts behind it.

    q, k, v = x Wqkv^T + b              moe_linear
    cache <- k turned, v; q turned      moe_kv_append
    a = softmax(q K^T scale) V          moe_prefix_attention
    h = a Wo^T + residual               moe_linear
    y = experts(norm(h))                MoELayer

The projections' weights may be in 8 bits (Rows8); their inputs then come in 8
bits too, from the norm ahead of them or brought there on the way:

    h = x + r;  z = norm(h)             moe_rms_norm      (RMSNorm)
    rows to 8 bits                      moe_quantize_rows
    y = x8 W8^T ...                     moe_linear_8bit

All calls run on one stream with no host synchronisation, so a step of a fixed
number of tokens and sequences can be captured in a CUDA graph: lengths,
positions, slots and page numbers are device arrays that a replay reads anew
(the prefix's length is a host number and stays as captured).  Norms: with
DecoderLayer.forward the one ahead of the attention side is the caller's, applied
to x, whose own value goes in as the residual, and the one ahead of the experts is
given to DecoderLayer; DecoderLayer.step has both.
"""
from __future__ import annotations

import dataclasses
from typing import Callable, List, Optional, Sequence

import numpy as np
import torch

from . import (E4M3, moe_check_waits, moe_kv_append, moe_linear, moe_linear_8bit, moe_linear_8bit_workspace_size,
               moe_linear_workspace_size, moe_prefix_attention, moe_prefix_attention_workspace_size, moe_quantize_rows,
               moe_rms_norm)


def rotation_table(max_position: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """cos | sin of p * base^(-2i / rot_dim) for p < max_position, fp32
    [max_position, rot_dim] (computed in fp64).  rot_dim is even."""
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError(f"rot_dim={rot_dim} must be even and not negative")
    f = base ** (-np.arange(0, rot_dim, 2, dtype=np.float64) / rot_dim)
    a = np.arange(max_position, dtype=np.float64)[:, None] * f
    return torch.from_numpy(np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32)).to(device)


@dataclasses.dataclass
class AttentionBatch:
    """One step's tokens: what moe_kv_append and moe_prefix_attention read
    besides the activations (device tensors; prefix_len a host number)."""
    positions: torch.Tensor     # int32 [T]
    slots: torch.Tensor         # int64 [T]
    cu_q: torch.Tensor          # int32 [B + 1]
    prefix_pages: torch.Tensor  # int32
    prefix_len: int
    page_table: torch.Tensor    # int32 [B, max_pages]
    seq_lens: torch.Tensor      # int32 [B], the step's tokens among them


def plan_batch(page_size: int, prefix_pages: Sequence[int], prefix_len: int, pages: Sequence[Sequence[int]],
               lens: Sequence[int], new: Sequence[int]):
    """Host arrays of a step in which sequence b, with lens[b] tokens of its own
    in the cache so far, adds new[b] tokens; pages[b] are its pages, enough for
    lens[b] + new[b] tokens.  Returns (positions, slots, cu_q, prefix_pages,
    page_table, seq_lens) as numpy arrays."""
    if not len(pages) == len(lens) == len(new):
        raise ValueError("pages, lens and new must have one entry per sequence")
    if page_size <= 0 or prefix_len < 0 or min(lens, default=0) < 0 or min(new, default=0) < 0:
        raise ValueError(f"page_size={page_size} must be positive, prefix_len={prefix_len} and the entries of lens and "
                         "new not negative")
    if prefix_len > len(prefix_pages) * page_size:
        raise ValueError(f"{len(prefix_pages)} prefix pages of {page_size} tokens hold no {prefix_len} tokens")
    pos: List[int] = []
    slots: List[int] = []
    table = np.zeros((len(pages), max([len(p) for p in pages] + [1])), np.int32)
    for b, (p, m, n) in enumerate(zip(pages, lens, new)):
        if m + n > len(p) * page_size:
            raise ValueError(f"sequence {b}: {len(p)} pages of {page_size} tokens hold no {m + n} tokens")
        table[b, :len(p)] = p
        for j in range(m, m + n):
            pos.append(prefix_len + j)
            slots.append(int(p[j // page_size]) * page_size + j % page_size)
    cu = np.concatenate(([0], np.cumsum(np.asarray(new, np.int64)))).astype(np.int32)
    total = np.asarray(lens, np.int64) + np.asarray(new, np.int64)
    return (np.asarray(pos, np.int32), np.asarray(slots, np.int64), cu, np.asarray(prefix_pages, np.int32), table,
            total.astype(np.int32))


def upload_batch(page_size: int, prefix_pages, prefix_len: int, pages, lens, new, device="cuda") -> AttentionBatch:
    """plan_batch on the device."""
    pos, slots, cu, pp, table, total = (torch.from_numpy(a).to(device) for a in
                                        plan_batch(page_size, prefix_pages, prefix_len, pages, lens, new))
    return AttentionBatch(pos, slots, cu, pp, prefix_len, table, total)


@dataclasses.dataclass
class Rows8:
    """Rows in 8 bits: q [n, K] (float8_e4m3fn) standing for q * scales[:, None]
    (fp32 [n])."""
    q: torch.Tensor
    scales: torch.Tensor

    @property
    def shape(self):
        return self.q.shape

    def __getitem__(self, rows: slice) -> "Rows8":
        return Rows8(self.q[rows], self.scales[rows])


def _rows8_like(n: int, K: int, device) -> Rows8:
    """Empty rows, whole 128 bytes apart (rows that start inside a sector cost a
    product up to a third)."""
    q = torch.empty(n, (K + 127) // 128 * 128, dtype=E4M3, device=device)[:, :K]
    return Rows8(q, torch.empty(n, dtype=torch.float32, device=device))


def quantize_rows(x: torch.Tensor, stream=None) -> Rows8:
    """x [n, K] (bf16, fp16 or fp32 on the device) in 8 bits: a projection's
    weights, once."""
    r = _rows8_like(x.shape[0], x.shape[1], x.device)
    moe_quantize_rows(x, r.q, r.scales, stream)
    return r


class RMSNorm:
    """h / sqrt(mean h^2 + eps) * weight with its buffers, for up to T_max tokens:
    weight [H] bf16 or fp16 on the device, kept by reference.  eight: results in 8
    bits (Rows8) instead of the weight's type.  Results are views of buffers that
    the next call overwrites."""

    def __init__(self, weight: torch.Tensor, eps: float, T_max: int, eight: bool = False):
        self.weight, self.eps, self.T_max, self.eight = weight, eps, T_max, eight
        self.H, self.dtype = weight.shape[0], weight.dtype
        self.h = torch.empty(T_max, self.H, dtype=weight.dtype, device=weight.device)
        self.y = _rows8_like(T_max, self.H, weight.device) if eight else torch.empty_like(self.h)

    def _out(self, T: int) -> dict:
        if T > self.T_max:
            raise ValueError(f"T={T} above T_max={self.T_max}")
        return dict(q=self.y.q[:T], scales=self.y.scales[:T]) if self.eight else dict(y=self.y[:T])

    def __call__(self, h, stream=None):
        """The norm of h [T, H]."""
        T = h.shape[0]
        moe_rms_norm(h, self.weight, self.eps, **self._out(T), stream=stream)
        return self.y[:T]

    def add(self, x, residual, stream=None):
        """(h, norm of h) for h = x + residual, rounded; x [T, H] fp32 or the
        weight's type."""
        T = x.shape[0]
        out = self._out(T)
        moe_rms_norm(x, self.weight, self.eps, residual=residual, h=self.h[:T], **out, stream=stream)
        return self.h[:T], self.y[:T]


class AttentionLayer:
    """Weights, buffers and the call sequence of one layer's attention side.

    w_qkv [(q_heads + 2 kv_heads) head_dim, H] with q, k and v rows in this
    order, b_qkv or None, w_out [H, q_heads head_dim], cos_sin from
    rotation_table (or None), k_cache / v_cache [pages, page_size, kv_heads,
    head_dim] (any strides with a contiguous last dimension); all bf16 or all
    fp16 on the device, kept by reference.  w_qkv and w_out may each be Rows8: that
    product then runs in 8 bits, and x may be Rows8 too.  T_max bounds a call's
    tokens."""

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, w_qkv, b_qkv, w_out, k_cache, v_cache, T_max: int,
                 cos_sin=None, interleaved: bool = False, scale: Optional[float] = None):
        self.q_heads, self.kv_heads, self.head_dim, self.T_max = q_heads, kv_heads, head_dim, T_max
        self.w_qkv, self.b_qkv, self.w_out = w_qkv, b_qkv, w_out
        self.k_cache, self.v_cache, self.cos_sin, self.interleaved = k_cache, v_cache, cos_sin, interleaved
        self.scale = head_dim ** -0.5 if scale is None else scale
        n_qkv, H = w_qkv.shape
        if n_qkv != (q_heads + 2 * kv_heads) * head_dim or tuple(w_out.shape) != (H, q_heads * head_dim):
            raise ValueError(f"w_qkv {tuple(w_qkv.shape)} / w_out {tuple(w_out.shape)} do not fit {q_heads} + 2 * "
                             f"{kv_heads} heads of {head_dim}")
        self.H, self.n_qkv = H, n_qkv
        dev, dt = k_cache.device, k_cache.dtype
        self.dtype = dt
        self.qkv = torch.empty(T_max, q_heads + 2 * kv_heads, head_dim, dtype=dt, device=dev)
        self.attn = torch.empty(T_max, q_heads, head_dim, dtype=dt, device=dev)
        self.lse = torch.empty(T_max, q_heads, dtype=torch.float32, device=dev)
        self.out = torch.empty(T_max, H, dtype=dt, device=dev)
        K = q_heads * head_dim
        # (8-bit products: their inputs' rows)
        self.x8 = _rows8_like(T_max, H, dev) if isinstance(w_qkv, Rows8) else None
        self.attn8 = _rows8_like(T_max, K, dev) if isinstance(w_out, Rows8) else None
        lin = max(f(T_max, n, k) for f in (moe_linear_workspace_size, moe_linear_8bit_workspace_size)
                  for n, k in ((n_qkv, H), (H, K)))
        self.ws = torch.zeros(lin, dtype=torch.uint8, device=dev)
        self.attn_ws = torch.zeros(moe_prefix_attention_workspace_size(T_max, q_heads, kv_heads, head_dim),
                                   dtype=torch.uint8, device=dev)

    def _project(self, x, w, y, bias, residual, rows: Optional[Rows8], stream):
        """y = x w^T + bias + residual; rows: where a 16-bit x goes to 8 bits."""
        if not isinstance(w, Rows8):
            if isinstance(x, Rows8):
                raise ValueError("8-bit rows need 8-bit weights")
            moe_linear(x, w, y, bias=bias, residual=residual, ws=self.ws, stream=stream)
            return
        if not isinstance(x, Rows8):
            r = rows[:x.shape[0]]
            moe_quantize_rows(x, r.q, r.scales, stream)
            x = r
        moe_linear_8bit(x.q, x.scales, w.q, w.scales, y, bias=bias, residual=residual, ws=self.ws, stream=stream)

    def forward(self, x, batch: AttentionBatch, residual=None, out=None, stream=None) -> torch.Tensor:
        """x [T, H] (or Rows8) -> residual + attention side of x (a view of self.out
        unless out is given); writes the step's keys and values into the cache."""
        T = x.shape[0]
        if T > self.T_max:
            raise ValueError(f"T={T} above T_max={self.T_max}")
        o = self.out[:T] if out is None else out
        qkv = self.qkv[:T]
        self._project(x, self.w_qkv, qkv.view(T, self.n_qkv), self.b_qkv, None, self.x8, stream)
        q, k, v = qkv.split((self.q_heads, self.kv_heads, self.kv_heads), 1)
        moe_kv_append(k, v, self.k_cache, self.v_cache, batch.positions, batch.slots, self.cos_sin,
                      interleaved=self.interleaved, q=q, q_out=q, stream=stream)
        moe_prefix_attention(q, self.k_cache, self.v_cache, batch.cu_q, batch.prefix_pages, batch.prefix_len,
                             batch.page_table, batch.seq_lens, self.scale, self.attn[:T], lse=self.lse[:T],
                             ws=self.attn_ws, stream=stream)
        self._project(self.attn[:T].view(T, self.q_heads * self.head_dim), self.w_out, o, None, residual, self.attn8, stream)
        return o

    def check(self) -> None:
        """Raises MoeError where a device-side wait of a forward since the last
        check has given up (waits for the current stream; see
        moe_check_waits)."""
        for ws, what in ((self.ws, "projections"), (self.attn_ws, "attention")):
            moe_check_waits(ws, what)


class DecoderLayer:
    """An AttentionLayer and the MoELayer behind it (bf16).  norm: what a model
    has between the two, h [T, H] -> the experts' tokens (bf16 [T, H],
    contiguous), without touching h (an RMSNorm, or any callable, whose result is
    looked at only when the attention side has run); None: h itself.  It runs with the
    call's stream as the current one.  norm_in: the RMSNorm ahead of the attention
    side, for step()."""

    def __init__(self, attention: AttentionLayer, moe, norm: Optional[Callable] = None, norm_in: Optional[RMSNorm] = None):
        if attention.H != moe.H:
            raise ValueError(f"hidden sizes differ: {attention.H} and {moe.H}")
        if norm is None and attention.dtype != torch.bfloat16:  # (the experts would take the bits for bf16)
            raise ValueError(f"the experts read bfloat16, the attention side writes {attention.dtype}")
        if norm_in is not None and (norm_in.H != attention.H or norm_in.dtype != attention.dtype):
            raise ValueError(f"norm_in: {norm_in.dtype} rows of {norm_in.H}, the attention side reads {attention.dtype} rows "
                             f"of {attention.H}")
        if isinstance(norm, RMSNorm) and (norm.eight or norm.H != moe.H or
                                          not norm.dtype == attention.dtype == torch.bfloat16):
            raise ValueError(f"norm: {'8-bit rows' if norm.eight else norm.dtype} of {norm.H}, the experts read bfloat16 rows "
                             f"of {moe.H}, the attention side writes {attention.dtype}")
        self.attention, self.moe, self.norm, self.norm_in = attention, moe, norm, norm_in

    def _fits(self, T: int, *others) -> None:
        """Before anything is written: T within the experts' and the norms' buffers."""
        norm = (("norm's", self.norm),) if isinstance(self.norm, RMSNorm) else ()
        for whose, n in (("the experts'", self.moe),) + norm + others:
            if T > n.T_max:
                raise ValueError(f"T={T} above {whose} T_max={n.T_max}")

    def forward(self, x, batch: AttentionBatch, residual=None, stream=None):
        """(h, y): h = residual + attention side of x ([T, H]), y = routed experts
        of norm(h) (fp32 [T, H]); the layer's result is h + y.  x may be Rows8 (see
        AttentionLayer)."""
        self._fits(x.shape[0])
        h = self.attention.forward(x, batch, residual, stream=stream)
        z = h
        if self.norm is not None:
            with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
                z = self.norm(h)
            if not isinstance(z, torch.Tensor) or z.dtype != torch.bfloat16 or z.shape != h.shape:
                raise ValueError(f"norm: expected bfloat16 {tuple(h.shape)}, got {getattr(z, 'dtype', type(z).__name__)} "
                                 f"{tuple(z.shape)}")
        return h, self.moe.forward(z, stream=stream, fresh=True)

    def step(self, h, y, batch: AttentionBatch, stream=None):
        """The layer behind another: (h, y) as that one returned them (y None ahead
        of the first layer, h then being the stream's 16-bit rows [T, H]).  The sum
        h + y, its norm (norm_in), the attention side on the stream h + y, norm and
        the experts.  Returns this layer's (h, y), as forward does."""
        if self.norm_in is None:
            raise ValueError("step needs norm_in")
        self._fits(h.shape[0], ("norm_in's", self.norm_in), ("the attention side's", self.attention))
        if y is None:
            z = self.norm_in(h, stream=stream)
        else:
            h, z = self.norm_in.add(y, h, stream=stream)
        return self.forward(z, batch, residual=h, stream=stream)
