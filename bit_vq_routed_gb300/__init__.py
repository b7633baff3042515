"""Python binding of libmoe_vq2.so, the GB300 (sm_103a) routed-expert VQ2 MoE
layer library.  Argument marshalling only: every step of the layer runs in
the library's CUDA kernels; PyTorch provides device memory and streams.

The functions carry the names of the C ABI in ``include/moe_vq2.h`` and take
CUDA tensors (any dtype of the right element size: bf16 activations as
``torch.bfloat16``, fp16 codebook/scales as ``torch.float16``, codes and
ue8m0 scales as ``torch.uint8``).  A non-zero status raises ``MoeError``
with the library's message.  There is no CPU or PyTorch fallback: if the
shared library cannot be built or loaded, the import of the functions fails.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import struct
import warnings
from typing import Optional, Sequence

import torch

from . import build as _build

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_CUDA = -3
MOE_ERR_NO_MEM = -4
MOE_ERR_WORKSPACE = -5
MOE_ERR_TIMEOUT = -6
MOE_ERR_MISMATCH = -7

MOE_FMT_VQ2 = 0
MOE_FMT_FP4 = 1
MOE_FUSED_SCATTER = 0
MOE_PER_PAIR = 1

MOE_DT_BF16 = 0
MOE_DT_F16 = 1
MOE_DT_F32 = 2
MOE_ACT_NONE = 0
MOE_ACT_RELU = 1
MOE_ACT_GELU = 2
MOE_ACT_GELU_TANH = 3
MOE_ACT_SILU = 4
MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1

LIB_PATH = _build.LIB


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"status {status}: {msg}")
        self.status = status


class _ExpertDesc(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int), ("codes", ctypes.c_void_p * 3), ("scales", ctypes.c_void_p * 3)]


class _KVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_stride", ctypes.c_int64 * 3),
                ("v_stride", ctypes.c_int64 * 3), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int)]


_KV_PACK = struct.Struct("@PP7q4i").pack  # the bytes of a moe_kv_cache
_APPEND_PACK = struct.Struct("@PP7q4iPPPP8qPPP5i4x").pack  # and of a moe_kv_append_args

_lib = None

EXPORTED = [
    "moe_version", "moe_last_error", "moe_vq2_pack", "moe_fp4_pack", "moe_slot_table_create",
    "moe_slot_table_set", "moe_slot_table_evict", "moe_slot_table_destroy", "moe_router_logits",
    "moe_route_topk", "moe_permute_workspace_size", "moe_permute",
    "moe_vq2_expert_ffn_workspace_size", "moe_vq2_expert_ffn", "moe_vq2_expert_ffn_noalloc", "moe_combine",
    "moe_launch_count", "moe_route_workspace_size", "moe_route", "moe_route_fresh", "moe_vq2_expert_ffn_combine",
    "moe_selftest", "moe_selftest_wait_timeout", "moe_expert_cache_slot_bytes", "moe_expert_cache_create", "moe_expert_cache_set_host",
    "moe_expert_cache_fetch", "moe_expert_cache_slot_of", "moe_expert_cache_stats", "moe_expert_cache_plan",
    "moe_expert_cache_destroy", "moe_expert_cache_set_host_image", "moe_cpu_pool_create", "moe_cpu_pool_threads",
    "moe_cpu_pool_destroy", "moe_cpu_expert_ffn", "moe_accumulate", "moe_slot_table_resident", "moe_vq2_pack_host",
    "moe_fp4_pack_host", "moe_confidence_gate", "moe_vq2_encoder_workspace_size", "moe_vq2_train_codebook", "moe_vq2_encode",
    "moe_linear_workspace_size", "moe_linear", "moe_kv_append", "moe_kv_append_packed", "moe_prefix_attention_workspace_size",
    "moe_prefix_attention", "moe_rms_norm", "moe_rms_norm_packed", "moe_quantize_rows", "moe_quantize_rows_packed",
    "moe_linear_8bit_workspace_size", "moe_linear_8bit", "moe_linear_8bit_packed", "moe_route_scored", "moe_route_scored_packed",
    "moe_route_tokens_scored",
]


def load(path: Optional[str] = None, build_if_stale: bool = True):
    """Loads (building it first if it is missing or older than its sources)
    the shared library and declares the C signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if path is None and build_if_stale:
        _build.build()
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with bit_vq_routed_gb300.build.build()")
    lib = ctypes.CDLL(p)
    P, I, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
    sig = {
        "moe_version": ([], I),
        "moe_last_error": ([], ctypes.c_char_p),
        "moe_vq2_pack": ([P, P, I, I, P, P, P], I),
        "moe_fp4_pack": ([P, P, I, I, P, P, P], I),
        "moe_slot_table_create": ([I, I, I, P, ctypes.POINTER(P)], I),
        "moe_slot_table_set": ([P, I, ctypes.POINTER(_ExpertDesc), P], I),
        "moe_slot_table_evict": ([P, I, P], I),
        "moe_slot_table_destroy": ([P], I),
        "moe_router_logits": ([P, P, P, P, I, I, I, P], I),
        "moe_route_topk": ([P, I, I, I, I, P, P, P], I),
        "moe_permute_workspace_size": ([I, I, I], Z),
        "moe_permute": ([P, I, I, I, P, P, P, P, Z, P], I),
        "moe_vq2_expert_ffn_workspace_size": ([I, I, I, I, I], Z),
        "moe_vq2_expert_ffn": ([P, P, P, P, P, I, I, I, P, P, P, Z, P], I),
        "moe_vq2_expert_ffn_noalloc": ([P, P, P, P, P, I, I, I, P, P, P], I),
        "moe_combine": ([P, P, P, P, I, I, I, P, P, P], I),
        "moe_launch_count": ([], ctypes.c_uint64),
        "moe_route_workspace_size": ([I, I, I], Z),
        "moe_route": ([P, P, P, I, I, I, I, I, P, P, P, P, P, P, P, Z, P], I),
        "moe_route_fresh": ([P, P, P, I, I, I, I, I, P, P, P, P, P, P, P, Z, P], I),
        "moe_vq2_expert_ffn_combine": ([P, P, P, P, P, P, I, I, P, P, P, P, P, Z, P], I),
        "moe_selftest": ([P], I),
        "moe_selftest_wait_timeout": ([P, P], I),
        "moe_expert_cache_slot_bytes": ([I, I, I], Z),
        "moe_expert_cache_create": ([P, P, Z, Z, ctypes.POINTER(P)], I),
        "moe_expert_cache_set_host": ([P, I, ctypes.POINTER(_ExpertDesc)], I),
        "moe_expert_cache_fetch": ([P, P, I, P, ctypes.POINTER(I), ctypes.POINTER(I), ctypes.POINTER(I)], I),
        "moe_expert_cache_slot_of": ([P, I], I),
        "moe_expert_cache_stats": ([P] + [ctypes.POINTER(ctypes.c_uint64)] * 4, I),
        "moe_expert_cache_plan": ([I, I, P, P, P, ctypes.c_uint64, P, I, P, P, ctypes.POINTER(I)], I),
        "moe_expert_cache_destroy": ([P, P], I),
        "moe_expert_cache_set_host_image": ([P, I, I, P], I),
        "moe_cpu_pool_create": ([I, ctypes.POINTER(P)], I),
        "moe_cpu_pool_threads": ([P], I),
        "moe_cpu_pool_destroy": ([P], I),
        "moe_cpu_expert_ffn": ([P, I, I, P, ctypes.POINTER(_ExpertDesc), I, P, P, P, P, I, I, P], I),
        "moe_accumulate": ([P, P, Z, P], I),
        "moe_slot_table_resident": ([P, I], I),
        "moe_vq2_pack_host": ([P, P, I, I, P, P], I),
        "moe_fp4_pack_host": ([P, P, I, I, P, P], I),
        "moe_confidence_gate": ([P, P, P, I, I, I, ctypes.c_float, P, P], I),
        "moe_vq2_encoder_workspace_size": ([I, I], Z),
        "moe_vq2_train_codebook": ([P, I, I, P, I, P, P, P, Z, P], I),
        "moe_vq2_encode": ([P, I, I, P, I, P, P, P, Z, P], I),
        "moe_linear_workspace_size": ([I, I, I], Z),
        "moe_linear": ([P, L, P, L, P, P, L, P, L, I, I, I, I, I, P, Z, P], I),
        "moe_kv_append_packed": ([P, P], I),
        "moe_kv_append": ([P, P, L, L, P, L, L, P, L, L, P, L, L, I, I, P, P, P, I, I, I, P], I),
        "moe_prefix_attention_workspace_size": ([I, I, I, I], Z),
        "moe_prefix_attention": ([P, P, L, L, I, I, P, I, P, L, P, L, I, P, ctypes.c_float, P, L, L, P, P, Z, P], I),
        "moe_rms_norm": ([P, L, I, P, L, P, L, P, ctypes.c_float, P, L, P, L, P, I, I, I, P], I),
        "moe_rms_norm_packed": ([P, P], I),
        "moe_linear_8bit_packed": ([P, P], I),
        "moe_route_scored_packed": ([P, P], I),
        "moe_quantize_rows_packed": ([P, P], I),
        "moe_quantize_rows": ([P, L, I, P, L, P, I, I, P], I),
        "moe_linear_8bit_workspace_size": ([I, I, I], Z),
        "moe_linear_8bit": ([P, L, P, P, L, P, P, P, L, P, L, I, I, I, I, I, P, Z, P], I),
        "moe_route_scored": ([P, I, I, I, P, P, P, P], I),
        "moe_route_tokens_scored": ([P, P, P, I, I, I, I, P, I, P, P, P, P, P, P, P, Z, P], I),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    if path is None:
        _load_binding(lib)
        _lib = lib
    return lib


# The short way to the smallest calls (csrc/binding.cpp): the status of a call that
# was made, or 1 where the arguments are for the functions below to look at.
def _look_again(*args) -> int:
    return 1


_quick_norm = _quick_rows = _quick_linear_8bit = _quick_route_scored = _look_again


def _load_binding(lib) -> None:
    """Without it (see build.binding_path) the functions below make the calls by way of
    ctypes, with the same results."""
    global _quick_norm, _quick_rows, _quick_linear_8bit, _quick_route_scored
    path = _build.binding_path()
    if not os.path.exists(path):
        return
    try:
        spec = importlib.util.spec_from_file_location("moe_binding", path)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        m.set_entry_points(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.moe_rms_norm_packed, lib.moe_quantize_rows_packed, lib.moe_linear_8bit_packed, lib.moe_route_scored_packed)))
    except Exception as e:
        warnings.warn(f"{os.path.basename(path)} does not load; its calls go by ctypes, which takes longer on the host: {e}",
                      RuntimeWarning, stacklevel=3)
        return
    _quick_norm, _quick_rows = m.rms_norm, m.quantize_rows
    _quick_linear_8bit, _quick_route_scored = m.linear_8bit, m.route_scored


def _check(status: int):
    if status != MOE_OK:
        raise MoeError(status, load().moe_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:  # (the handle alone: building a Stream object costs 3 us)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ------------------------------------------------------------------ formats

def moe_vq2_pack(codes, scales, packed_codes, packed_scales, stream=None):
    rows, G = codes.shape
    _check(load().moe_vq2_pack(_ptr(codes), _ptr(scales), rows, 4 * G, _ptr(packed_codes),
                               _ptr(packed_scales), _stream(stream)))


def moe_fp4_pack(codes, scales, packed_codes, packed_scales, stream=None):
    rows, nb = codes.shape
    _check(load().moe_fp4_pack(_ptr(codes), _ptr(scales), rows, 2 * nb, _ptr(packed_codes),
                               _ptr(packed_scales), _stream(stream)))


class SlotTable:
    """moe_slot_table_create / _set / _evict / _destroy.  Keeps references to
    the tensors of every set entry so they outlive the table's use of them."""

    def __init__(self, num_experts: int, H: int, I: int, codebook: torch.Tensor):
        self.lib = load()
        self.codebook = codebook
        self.E, self.H, self.I = num_experts, H, I
        h = ctypes.c_void_p()
        _check(self.lib.moe_slot_table_create(num_experts, H, I, _ptr(codebook), ctypes.byref(h)))
        self.handle = h
        self._keep = {}

    def set(self, expert_id: int, fmt: int, codes: Sequence[torch.Tensor], scales: Sequence[torch.Tensor],
            stream=None):
        d = _ExpertDesc()
        d.format = fmt
        for m in range(3):
            d.codes[m] = _ptr(codes[m])
            d.scales[m] = _ptr(scales[m])
        _check(self.lib.moe_slot_table_set(self.handle, expert_id, ctypes.byref(d), _stream(stream)))
        self._keep[expert_id] = (list(codes), list(scales))

    def evict(self, expert_id: int, stream=None):
        _check(self.lib.moe_slot_table_evict(self.handle, expert_id, _stream(stream)))

    def destroy(self):
        if self.handle is not None:
            _check(self.lib.moe_slot_table_destroy(self.handle))
            self.handle = None
            self._keep.clear()

    def __del__(self):
        try:
            if self.handle is not None and torch.cuda.is_initialized():
                torch.cuda.synchronize()
                self.destroy()
        except Exception:
            pass


# ------------------------------------------------------------------ hot path

def moe_router_logits(x, w_router, bias, logits, stream=None):
    T, H = x.shape
    E = w_router.shape[0]
    _check(load().moe_router_logits(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(logits), T, H, E,
                                    _stream(stream)))


def moe_route_topk(logits, k: int, renormalize: int, ids, weights, stream=None):
    T, E = logits.shape
    _check(load().moe_route_topk(_ptr(logits), T, E, k, renormalize, _ptr(ids), _ptr(weights),
                                 _stream(stream)))


def moe_permute_workspace_size(T: int, k: int, E: int) -> int:
    return load().moe_permute_workspace_size(T, k, E)


def moe_permute(ids, E: int, expert_offsets, sorted_pair, pair_to_sorted, ws=None, stream=None):
    T, k = ids.shape
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().moe_permute(_ptr(ids), T, k, E, _ptr(expert_offsets), _ptr(sorted_pair),
                              _ptr(pair_to_sorted), _ptr(ws), nbytes, _stream(stream)))


def moe_vq2_expert_ffn_workspace_size(T: int, k: int, E: int, H: int, I: int) -> int:
    return load().moe_vq2_expert_ffn_workspace_size(T, k, E, H, I)


def moe_vq2_expert_ffn(table: SlotTable, x, expert_offsets, sorted_pair, weights, k: int, mode: int,
                       out, pair_status, ws, stream=None):
    T = x.shape[0]
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().moe_vq2_expert_ffn(table.handle, _ptr(x), _ptr(expert_offsets), _ptr(sorted_pair),
                                     _ptr(weights), T, k, mode, _ptr(out), _ptr(pair_status), _ptr(ws),
                                     nbytes, _stream(stream)))


MOE_NOALLOC_SCRATCH_BYTES = 64 << 20


def moe_vq2_expert_ffn_noalloc(table: SlotTable, x, expert_offsets, sorted_pair, weights, k: int, mode: int,
                               out, pair_status, stream=None):
    """moe_vq2_expert_ffn without a workspace argument, for callers that cannot
    allocate device memory: the library's fixed MOE_NOALLOC_SCRATCH_BYTES
    device array serves as scratch (shared by every call on a device, so
    calls must not overlap on the GPU)."""
    T = x.shape[0]
    _check(load().moe_vq2_expert_ffn_noalloc(table.handle, _ptr(x), _ptr(expert_offsets), _ptr(sorted_pair),
                                             _ptr(weights), T, k, mode, _ptr(out), _ptr(pair_status),
                                             _stream(stream)))


def moe_combine(ypair, pair_to_sorted, weights, pair_status, k: int, out_f32=None, out_bf16=None,
                stream=None):
    T = weights.shape[0]
    H = ypair.shape[1]
    _check(load().moe_combine(_ptr(ypair), _ptr(pair_to_sorted), _ptr(weights), _ptr(pair_status), T, k,
                              H, _ptr(out_f32), _ptr(out_bf16), _stream(stream)))




def moe_launch_count() -> int:
    """Kernel launches the library has issued since it was loaded (a launch
    inside a stream capture counts once)."""
    return int(load().moe_launch_count())


def moe_selftest(stream=None) -> None:
    """Boot self-check of the library on the current device: runs a tiny
    layer through every kernel family and compares with stored CPU-reference
    results.  Synchronises the stream; raises MoeError (status
    MOE_ERR_MISMATCH for a wrong result) on failure."""
    _check(load().moe_selftest(_stream(stream)))


def moe_selftest_wait_timeout(stream=None) -> dict:
    """Self-check of the kernels' bounded-wait pattern: two waits on mbarriers
    that nothing completes give up, record their codes and return.  Raises
    MoeError if they do not; returns the codes and each wait's microseconds."""
    codes = (ctypes.c_int * 6)()
    _check(load().moe_selftest_wait_timeout(codes, _stream(stream)))
    return dict(codes=(codes[0], codes[1]), gave_up=(codes[2] == 0, codes[3] == 0), us=(codes[4], codes[5]))


def moe_route_workspace_size(T: int, k: int, E: int) -> int:
    return int(load().moe_route_workspace_size(T, k, E))


def moe_route(x, w_router, bias, k: int, renormalize: int, logits, ids, weights, expert_offsets, sorted_pair,
              pair_to_sorted, ws, stream=None, fresh: bool = False):
    """Router logits, top-k softmax and permutation in one call (one kernel
    for small batches).  ws: a zero-filled device buffer of at least
    moe_route_workspace_size bytes, left zeroed by the call.  fresh: x may be
    written by the kernel enqueued just before (moe_route_fresh); without it
    x has to be complete by then."""
    T, H = x.shape
    E = w_router.shape[0]
    call = load().moe_route_fresh if fresh else load().moe_route
    _check(call(_ptr(x), _ptr(w_router), _ptr(bias), T, H, E, k, renormalize, _ptr(logits), _ptr(ids),
                _ptr(weights), _ptr(expert_offsets), _ptr(sorted_pair), _ptr(pair_to_sorted), _ptr(ws),
                ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream)))


def moe_vq2_expert_ffn_combine(table: "SlotTable", x, expert_offsets, sorted_pair, pair_to_sorted, weights, k: int,
                               ypair, pair_status, out_f32=None, out_bf16=None, ws=None, stream=None):
    """moe_vq2_expert_ffn (per-pair mode) and then moe_combine in one call
    (for single-token calls the combine runs inside the expert kernels)."""
    T = x.shape[0]
    _check(load().moe_vq2_expert_ffn_combine(table.handle, _ptr(x), _ptr(expert_offsets), _ptr(sorted_pair),
                                             _ptr(pair_to_sorted), _ptr(weights), T, k, _ptr(ypair),
                                             _ptr(pair_status), _ptr(out_f32), _ptr(out_bf16), _ptr(ws),
                                             ws.numel() * ws.element_size() if ws is not None else 0,
                                             _stream(stream)))


# ------------------------------------------------------------------ expert cache

def moe_expert_cache_slot_bytes(H: int, I: int, fmt: int) -> int:
    """Bytes of one cache slot for an expert of format fmt."""
    return int(load().moe_expert_cache_slot_bytes(H, I, fmt))


def moe_expert_cache_plan(num_experts: int, slot_expert, counts, last_step, step: int, request):
    """Host-only planning step of the expert cache.  slot_expert (int32),
    counts and last_step (uint64) are numpy arrays updated in place; returns
    (fill_slot, evicted, n_unplaced) for the requests."""
    import numpy as np
    for a, dt in ((slot_expert, np.int32), (counts, np.uint64), (last_step, np.uint64)):
        if not (isinstance(a, np.ndarray) and a.dtype == dt and a.flags.c_contiguous):
            raise ValueError(f"expected a contiguous numpy {dt.__name__} array")
    req = np.ascontiguousarray(request, dtype=np.int32)
    fill = np.empty(req.size, np.int32)
    ev = np.empty(req.size, np.int32)
    left = ctypes.c_int(0)
    vp = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    _check(load().moe_expert_cache_plan(num_experts, slot_expert.size, vp(slot_expert), vp(counts), vp(last_step),
                                        step, vp(req), req.size, vp(fill), vp(ev), ctypes.byref(left)))
    return fill, ev, left.value


def _host_ptr(t: torch.Tensor) -> int:
    if t.is_cuda or not t.is_pinned():
        raise ValueError("expected a page-locked (pinned) host tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


class ExpertCache:
    """moe_expert_cache_*: slot-table entries filled on a miss from pinned
    host copies of the experts' packed buffers, into slots of a device pool
    (a uint8 CUDA tensor this object keeps).  Keeps references to the host
    tensors it was given."""

    def __init__(self, table: SlotTable, pool: torch.Tensor, slot_bytes: int):
        self.lib = load()
        self.table, self.pool, self.slot_bytes = table, pool, slot_bytes
        h = ctypes.c_void_p()
        _check(self.lib.moe_expert_cache_create(table.handle, _ptr(pool), pool.numel() * pool.element_size(),
                                                slot_bytes, ctypes.byref(h)))
        self.handle = h
        self.num_slots = pool.numel() * pool.element_size() // slot_bytes
        self._host = {}

    def set_host(self, expert_id: int, fmt: int, codes: Sequence[torch.Tensor], scales: Sequence[torch.Tensor]):
        H, I = self.table.H, self.table.I
        for m in range(3):  # the packed sizes the fetch copies (the C side trusts them)
            rows, K = (H, I) if m == 2 else (I, H)
            want = (rows * K // 4, rows * K // 128 * 2) if fmt == MOE_FMT_VQ2 else (rows * K // 2, rows * K // 32)
            got = (codes[m].numel() * codes[m].element_size(), scales[m].numel() * scales[m].element_size())
            if got != want:
                raise ValueError(f"expert {expert_id} matrix {m}: {got} bytes of codes/scales, expected {want}")
        d = _ExpertDesc()
        d.format = fmt
        for m in range(3):
            d.codes[m] = _host_ptr(codes[m])
            d.scales[m] = _host_ptr(scales[m])
        _check(self.lib.moe_expert_cache_set_host(self.handle, expert_id, ctypes.byref(d)))
        self._host[expert_id] = (list(codes), list(scales))

    def set_host_image(self, expert_id: int, fmt: int, image: torch.Tensor):
        """One pinned uint8 block in the slot's layout (host_expert_image):
        fetched with one copy."""
        want = moe_expert_cache_slot_bytes(self.table.H, self.table.I, fmt)
        if image.numel() * image.element_size() != want:
            raise ValueError(f"expert {expert_id}: image of {image.numel() * image.element_size()} bytes, "
                             f"expected {want}")
        _check(self.lib.moe_expert_cache_set_host_image(self.handle, expert_id, fmt, _host_ptr(image)))
        self._host[expert_id] = image

    def fetch(self, experts, stream=None) -> dict:
        """One step: makes the named experts resident (see the C header for
        the eviction rule).  Returns n_fetched, n_unplaced and recapture."""
        import numpy as np
        ids = np.ascontiguousarray(np.asarray(experts).ravel(), dtype=np.int32)
        nf, nu, rc = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
        _check(self.lib.moe_expert_cache_fetch(self.handle, ids.ctypes.data_as(ctypes.c_void_p), ids.size,
                                               _stream(stream), ctypes.byref(nf), ctypes.byref(nu),
                                               ctypes.byref(rc)))
        return dict(n_fetched=nf.value, n_unplaced=nu.value, recapture=bool(rc.value))

    def slot_of(self, expert_id: int) -> int:
        return int(self.lib.moe_expert_cache_slot_of(self.handle, expert_id))

    def stats(self) -> dict:
        v = [ctypes.c_uint64(0) for _ in range(4)]
        _check(self.lib.moe_expert_cache_stats(self.handle, *[ctypes.byref(x) for x in v]))
        return dict(hits=v[0].value, misses=v[1].value, unplaced=v[2].value, bytes_fetched=v[3].value)

    def destroy(self, stream=None):
        if self.handle is not None:
            h, self.handle = self.handle, None
            if self.table.handle is not None:  # (the table's entries die with the table)
                _check(self.lib.moe_expert_cache_destroy(h, _stream(stream)))

    def __del__(self):
        try:
            if self.handle is not None and torch.cuda.is_initialized():
                self.destroy()
                torch.cuda.synchronize()
        except Exception:
            pass


# ------------------------------------------------------------------ host CPU path

def _np_ptr(a, dtype=None):
    """(pointer, keep-alive) of a contiguous host array: a numpy array or a
    CPU torch tensor."""
    import numpy as np
    if isinstance(a, torch.Tensor):
        if a.is_cuda:
            raise ValueError("expected a host array")
        a = a.contiguous()
        return a.data_ptr(), a
    arr = np.ascontiguousarray(a if dtype is None else np.asarray(a, dtype=dtype))
    return arr.ctypes.data, arr


def moe_vq2_pack_host(codes, scales):
    """Packs a logical VQ2 matrix on the host (uint8 [rows, K/4], fp16 bits
    [rows, K/4/32]) into the slot layout; returns (packed codes, packed
    scales) as numpy arrays of the same shapes and types."""
    import numpy as np
    c = np.ascontiguousarray(codes, dtype=np.uint8)
    sc = np.ascontiguousarray(scales, dtype=np.uint16)
    rows, G = c.shape
    pc, ps = np.empty_like(c), np.empty_like(sc)
    _check(load().moe_vq2_pack_host(c.ctypes.data, sc.ctypes.data, rows, 4 * G, pc.ctypes.data, ps.ctypes.data))
    return pc, ps


def moe_fp4_pack_host(codes, scales):
    """The same for a logical FP4 matrix (uint8 [rows, K/2], uint8 [rows, K/32])."""
    import numpy as np
    c = np.ascontiguousarray(codes, dtype=np.uint8)
    sc = np.ascontiguousarray(scales, dtype=np.uint8)
    rows, nb = c.shape
    pc, ps = np.empty_like(c), np.empty_like(sc)
    _check(load().moe_fp4_pack_host(c.ctypes.data, sc.ctypes.data, rows, 2 * nb, pc.ctypes.data, ps.ctypes.data))
    return pc, ps


def host_pack_expert(fmt: int, codes: Sequence, scales: Sequence):
    """One expert's three matrices packed on the host: (fmt, [codes x3], [scales x3])."""
    pack = moe_vq2_pack_host if fmt == MOE_FMT_VQ2 else moe_fp4_pack_host
    pcs, pss = [], []
    for m in range(3):
        pc, ps = pack(codes[m], scales[m])
        pcs.append(pc)
        pss.append(ps)
    return fmt, pcs, pss


class CpuPool:
    """moe_cpu_pool: host threads for moe_cpu_expert_ffn (threads <= 0: all)."""

    def __init__(self, threads: int = 0):
        self.lib = load()
        h = ctypes.c_void_p()
        _check(self.lib.moe_cpu_pool_create(threads, ctypes.byref(h)))
        self.handle = h

    @property
    def threads(self) -> int:
        return int(self.lib.moe_cpu_pool_threads(self.handle))

    def close(self):
        if self.handle is not None:
            h, self.handle = self.handle, None
            _check(self.lib.moe_cpu_pool_destroy(h))

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class HostExperts:
    """The moe_expert_desc array of host-resident packed experts that
    moe_cpu_expert_ffn reads: entry e is (fmt, [codes x3], [scales x3]) host
    arrays (host_pack_expert) or None.  Keeps the arrays alive."""

    def __init__(self, E: int):
        self.E = E
        self.descs = (_ExpertDesc * E)()
        self._keep = {}

    def set(self, e: int, fmt: int, codes: Sequence, scales: Sequence):
        d = self.descs[e]
        d.format = fmt
        keep = []
        for m in range(3):
            pc, kc = _np_ptr(codes[m])
            ps, ks = _np_ptr(scales[m])
            d.codes[m] = pc
            d.scales[m] = ps
            keep += [kc, ks]
        self._keep[e] = keep


def moe_cpu_expert_ffn(pool: CpuPool, H: int, I: int, codebook, experts: HostExperts, x, ids, weights,
                       gpu_status, k: int, out=None):
    """The remainder of the combine over the pairs with gpu_status 0,
    computed on the host (see the C header).  x: host bf16 bits [T, H];
    ids int32 / weights fp32 [T, k]; gpu_status uint8 [T*k]; out: host fp32
    [T, H] (allocated when None).  Returns out."""
    import numpy as np
    xp, xk = _np_ptr(x, np.uint16)
    ip, ik = _np_ptr(ids, np.int32)
    wp, wk = _np_ptr(weights, np.float32)
    sp, sk = _np_ptr(gpu_status, np.uint8)
    cp, ck = _np_ptr(codebook, np.uint16)
    T = int(np.prod(xk.shape)) // H
    if out is None:
        out = np.empty((T, H), np.float32)
    op, ok = _np_ptr(out)
    _check(load().moe_cpu_expert_ffn(pool.handle, H, I, cp, experts.descs, experts.E, xp, ip, wp, sp, T, k, op))
    return out


def moe_accumulate(dst, src, stream=None):
    """dst += src on the device (fp32 CUDA tensors of equal size)."""
    if dst.numel() != src.numel():
        raise ValueError("moe_accumulate: sizes differ")
    _check(load().moe_accumulate(_ptr(dst), _ptr(src), dst.numel(), _stream(stream)))


def moe_slot_table_resident(table: "SlotTable", expert_id: int) -> bool:
    r = int(load().moe_slot_table_resident(table.handle, expert_id))
    if r < 0:
        _check(r)
    return r == 1


def moe_confidence_gate(table: "SlotTable", ids, weights, E: int, tau: float, gated_ids, stream=None):
    """gated_ids = ids + E where weights >= tau and the table holds entry
    E + id (the expert's FP4 weights), ids elsewhere (see the C header)."""
    T, k = ids.shape
    _check(load().moe_confidence_gate(table.handle, _ptr(ids), _ptr(weights), T, k, E, tau, _ptr(gated_ids),
                                      _stream(stream)))


# ------------------------------------------------------------------ attention side

_DTYPES = {torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16}

# These calls are short beside their arguments' handling at decode sizes, so
# each looks at its tensors in one condition and names the fault only where
# there is one.


def _fault(dtype, *tensors):
    """Raises ValueError for the first of (name, tensor, shape) that is not a
    CUDA tensor of that type and shape with a contiguous last dimension."""
    if dtype not in _DTYPES:
        raise ValueError(f"expected bfloat16 or float16, got {dtype}")
    for what, t, shape in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{what}: expected a CUDA tensor")
        if t.dtype != dtype:
            raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{what}: expected a contiguous last dimension")


def _ints_ptr(t: torch.Tensor, n: int, dtype, what: str):
    """Pointer of a contiguous CUDA vector of n elements."""
    if not (t.is_cuda and t.dtype == dtype and t.shape == (n,) and (n <= 1 or t.stride(0) == 1)):
        raise ValueError(f"{what}: expected a contiguous CUDA tensor {dtype} ({n},), got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")
    return t.data_ptr()


def _ws(ws: Optional[torch.Tensor]):
    """(pointer, bytes) of a workspace."""
    if ws is None:
        return None, 0
    return _ptr(ws), ws.nbytes


def moe_check_waits(ws: torch.Tensor, what: str = "workspace") -> None:
    """Raises MoeError (MOE_ERR_TIMEOUT) where a device-side wait of a call with
    this workspace (moe_linear, moe_prefix_attention) has given up since the
    last look: that call's results are not to be used.  Clears the note.  Reads
    the device behind the work of the current stream and waits for it."""
    word = ws[8:12].view(torch.int32)
    code = int(word.item())
    if code != 0:
        word.zero_()
        raise MoeError(MOE_ERR_TIMEOUT, f"{what}: a device-side wait gave up (code {code}); results are not valid")


def moe_linear_workspace_size(T: int, N: int, K: int) -> int:
    return int(load().moe_linear_workspace_size(T, N, K))


def moe_linear(x, w, y, bias=None, act: int = MOE_ACT_NONE, residual=None, ws=None, stream=None):
    """y[T, N] = act(x[T, K] w[N, K]^T + bias[N]) + residual[T, N] (see the C
    header).  Rows may be strided; residual may be y.  ws: a zero-filled
    device buffer of at least moe_linear_workspace_size bytes."""
    T, K = x.shape
    N = w.shape[0]
    dt = x.dtype
    sx, sw, sy = x.stride(), w.stride(), y.stride()
    if not (dt in _DTYPES and x.is_cuda and w.is_cuda and y.is_cuda and w.dtype == dt and y.dtype == dt and
            w.shape == (N, K) and y.shape == (T, N) and sx[1] == 1 and sw[1] == 1 and sy[1] == 1):
        _fault(dt, ("x", x, (T, K)), ("w", w, (N, K)), ("y", y, (T, N)))
    bp = rp = None
    ldr = 0
    if bias is not None:
        if not (bias.is_cuda and bias.dtype == dt and bias.shape == (N,) and bias.stride(0) == 1):
            _fault(dt, ("bias", bias, (N,)))
        bp = bias.data_ptr()
    if residual is not None:
        if not (residual.is_cuda and residual.dtype == dt and residual.shape == (T, N) and residual.stride(1) == 1):
            _fault(dt, ("residual", residual, (T, N)))
        rp, ldr = residual.data_ptr(), residual.stride(0)
    wp, wn = _ws(ws)
    _check(load().moe_linear(x.data_ptr(), sx[0], w.data_ptr(), sw[0], bp, rp, ldr, y.data_ptr(), sy[0], T, N, K,
                             _DTYPES[dt], act, wp, wn, _stream(stream)))


def _kv_cache(k_cache: torch.Tensor, v_cache: torch.Tensor) -> bytes:
    """The moe_kv_cache of two tensors [num_pages, page_size, kv_heads,
    head_dim] (any strides with a contiguous last dimension: a cache kept as
    [num_pages, kv_heads, page_size, head_dim] is passed as its
    transpose(1, 2))."""
    shape, dt = k_cache.shape, k_cache.dtype
    n, p, h, D = shape
    a, b = k_cache.stride(), v_cache.stride()
    if not (k_cache.is_cuda and v_cache.is_cuda and dt in _DTYPES and v_cache.dtype == dt and v_cache.shape == shape and
            a[3] == 1 and b[3] == 1):
        _fault(dt, ("k_cache", k_cache, shape), ("v_cache", v_cache, shape))
    return _KV_PACK(k_cache.data_ptr(), v_cache.data_ptr(), a[0], a[1], a[2], b[0], b[1], b[2], n, p, h, D, _DTYPES[dt])


def moe_kv_append(k, v, k_cache, v_cache, positions, slots, cos_sin=None, interleaved: bool = False, q=None,
                  q_out=None, stream=None):
    """Writes k, v [T, kv_heads, head_dim] into the cache's slots (int64 [T],
    negative: padding), the keys turned by their positions (int32 [T]) with
    cos_sin (fp32 [max_position, rot_dim]; None: no rotation), and the turned
    q [T, q_heads, head_dim] into q_out (which may be q).  See the C header."""
    n, p, h, D = size = k_cache.shape
    T = k.shape[0]
    row = (T, h, D)
    dt = k_cache.dtype
    a, b, sk, sv = k_cache.stride(), v_cache.stride(), k.stride(), v.stride()
    if not (k_cache.is_cuda and v_cache.is_cuda and k.is_cuda and v.is_cuda and dt in _DTYPES and
            v_cache.dtype == dt and k.dtype == dt and v.dtype == dt and v_cache.shape == size and k.shape == row and
            v.shape == row and a[3] == 1 and b[3] == 1 and sk[2] == 1 and sv[2] == 1):
        _fault(dt, ("k_cache", k_cache, size), ("v_cache", v_cache, size), ("k", k, row), ("v", v, row))
    rot = maxp = cp = pp = 0
    if cos_sin is not None:
        maxp, rot = cos_sin.shape
        if not (cos_sin.is_cuda and cos_sin.dtype == torch.float32 and cos_sin.is_contiguous()):
            raise ValueError("cos_sin: expected a contiguous fp32 CUDA tensor")
        cp, pp = cos_sin.data_ptr(), _ints_ptr(positions, T, torch.int32, "positions")
    qh = q0 = q1 = qp = o0 = o1 = op = 0
    if q is not None:
        if q_out is None:
            raise ValueError("q_out is missing")
        qh = q.shape[1]
        row = (T, qh, D)
        sq, so = q.stride(), q_out.stride()
        if not (q.is_cuda and q_out.is_cuda and q.dtype == dt and q_out.dtype == dt and q.shape == row and
                q_out.shape == row and sq[2] == 1 and so[2] == 1):
            _fault(dt, ("q", q, row), ("q_out", q_out, row))
        q0, q1, qp, o0, o1, op = sq[0], sq[1], q.data_ptr(), so[0], so[1], q_out.data_ptr()
    # (26 arguments take ctypes 2 us, one 0.2)
    args = _APPEND_PACK(k_cache.data_ptr(), v_cache.data_ptr(), a[0], a[1], a[2], b[0], b[1], b[2], n, p, h, D,
                        _DTYPES[dt], k.data_ptr(), v.data_ptr(), qp, op, sk[0], sk[1], sv[0], sv[1], q0, q1, o0, o1,
                        pp, _ints_ptr(slots, T, torch.int64, "slots"), cp, qh, T, maxp, rot, interleaved)
    _check(load().moe_kv_append_packed(args, _stream(stream)))


def moe_prefix_attention_workspace_size(T: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(load().moe_prefix_attention_workspace_size(T, q_heads, kv_heads, head_dim))


def moe_prefix_attention(q, k_cache, v_cache, cu_q, prefix_pages, prefix_len: int, page_table, seq_lens,
                         scale: float, out, lse=None, ws=None, stream=None):
    """Attention of q [T, q_heads, head_dim], sequence b's tokens being
    cu_q[b] .. cu_q[b+1]-1, over the prefix_len tokens of prefix_pages (int32)
    that all sequences share and, causally, over each sequence's own
    seq_lens[b] tokens in the pages of page_table[b] (int32 [B, max_pages],
    rows may be strided).  Writes out [T, q_heads, head_dim] and lse (fp32
    [T, q_heads], optional).  ws: a zero-filled device buffer of at least
    moe_prefix_attention_workspace_size bytes.  See the C header."""
    T, qh, D = q.shape
    cache = _kv_cache(k_cache, v_cache)
    dt = k_cache.dtype
    sq, so = q.stride(), out.stride()
    if not (q.is_cuda and out.is_cuda and q.dtype == dt and out.dtype == dt and D == k_cache.shape[3] and
            out.shape == (T, qh, D) and sq[2] == 1 and so[2] == 1):
        _fault(dt, ("q", q, (T, qh, k_cache.shape[3])), ("out", out, (T, qh, D)))
    B, max_pages = page_table.shape
    st = page_table.stride()
    if not (page_table.is_cuda and page_table.dtype == torch.int32 and (st[1] == 1 or max_pages <= 1)):
        raise ValueError("page_table: expected an int32 CUDA tensor with contiguous rows")
    pages = None
    if prefix_len > 0:
        need = -(-prefix_len // k_cache.shape[1])
        if prefix_pages.dim() != 1 or prefix_pages.shape[0] < need:
            raise ValueError(f"prefix_pages: {need} pages needed, got {tuple(prefix_pages.shape)}")
        pages = _ints_ptr(prefix_pages, prefix_pages.shape[0], torch.int32, "prefix_pages")
    lp = None
    if lse is not None:
        if not (lse.is_cuda and lse.dtype == torch.float32 and lse.shape == (T, qh) and lse.is_contiguous()):
            raise ValueError(f"lse: expected a contiguous fp32 CUDA tensor {(T, qh)}")
        lp = lse.data_ptr()
    wp, wn = _ws(ws)
    _check(load().moe_prefix_attention(
        cache, q.data_ptr(), sq[0], sq[1], qh, T, _ints_ptr(cu_q, B + 1, torch.int32, "cu_q"), B, pages, prefix_len,
        page_table.data_ptr(), st[0], max_pages, _ints_ptr(seq_lens, B, torch.int32, "seq_lens"), scale,
        out.data_ptr(), so[0], so[1], lp, wp, wn, _stream(stream)))


# ------------------------------------------------------------------ norms, 8-bit products, choice by score

E4M3 = torch.float8_e4m3fn
_F32 = torch.float32
_NORM_PACK = struct.Struct("@7P5qf4i4x").pack  # the bytes of a moe_rms_norm_args
_ROWS_PACK = struct.Struct("@PPPqq3i4x").pack  # of a moe_quantize_rows_args
_LINEAR8_PACK = struct.Struct("@8P4qN5i4x").pack  # and of a moe_linear_8bit_args
_X_DTYPES = {torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16, torch.float32: MOE_DT_F32}


def _rows_fault(*tensors):
    """Raises ValueError for the first of (name, tensor, types, shape) that is not
    a CUDA tensor of one of those types and of that shape, with a contiguous last
    dimension."""
    for what, t, types, shape in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{what}: expected a CUDA tensor")
        if t.dtype not in types:
            raise ValueError(f"{what}: expected {' or '.join(str(d) for d in types)}, got {t.dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{what}: expected a contiguous last dimension")


def moe_rms_norm(x, weight, eps: float, residual=None, h=None, y=None, q=None, scales=None, dtype=None, stream=None):
    """h = x + residual, rounded; y = h / sqrt(mean h^2 + eps) * weight [H]
    (None: ones), as y [T, H] and/or in 8 bits as q (float8_e4m3fn [T, H]) with
    scales (fp32 [T]).  x [T, H] has the others' type, or is fp32.  Rows may be
    strided; h may be residual or None.  dtype: the type, where no tensor but x
    tells it.  See the C header."""
    status = _quick_norm(x, weight, eps, residual, h, y, q, scales, stream)
    if status != 1:
        if status:
            _check(status)
        return
    row = x.shape
    T, H = row
    xd, sx = x.dtype, x.stride()
    dt = weight.dtype if weight is not None else residual.dtype if residual is not None else y.dtype if y is not None else \
        dtype if dtype is not None else xd if xd != _F32 else torch.bfloat16
    wp = rp = hp = yp = qp = sp = ldr = ldh = ldy = ldq = 0
    if not (dt in _DTYPES and x.is_cuda and (xd == dt or xd == _F32) and sx[1] == 1):
        if dt not in _DTYPES:
            raise ValueError(f"expected bfloat16 or float16, got {dt}")
        _rows_fault(("x", x, (dt, _F32), row))
    if weight is not None:
        if not (weight.is_cuda and weight.shape == (H,) and weight.is_contiguous()):
            _rows_fault(("weight", weight, (dt,), (H,)))
        wp = weight.data_ptr()
    if residual is not None:
        st = residual.stride()
        if not (residual.is_cuda and residual.dtype == dt and residual.shape == row and st[1] == 1):
            _rows_fault(("residual", residual, (dt,), row))
        rp, ldr = residual.data_ptr(), st[0]
    if h is not None:
        st = h.stride()
        if not (h.is_cuda and h.dtype == dt and h.shape == row and st[1] == 1):
            _rows_fault(("h", h, (dt,), row))
        hp, ldh = h.data_ptr(), st[0]
    if y is not None:
        st = y.stride()
        if not (y.is_cuda and y.dtype == dt and y.shape == row and st[1] == 1):
            _rows_fault(("y", y, (dt,), row))
        yp, ldy = y.data_ptr(), st[0]
    if q is not None:
        st = q.stride()
        if not (q.is_cuda and q.dtype == E4M3 and q.shape == row and st[1] == 1):
            _rows_fault(("q", q, (E4M3,), row))
        qp, ldq = q.data_ptr(), st[0]
    if scales is not None:
        if not (scales.is_cuda and scales.dtype == _F32 and scales.shape == (T,) and scales.is_contiguous()):
            _rows_fault(("scales", scales, (_F32,), (T,)))
        sp = scales.data_ptr()
    args = _NORM_PACK(x.data_ptr(), rp, wp, hp, yp, qp, sp, sx[0], ldr, ldh, ldy, ldq, eps, T, H, _X_DTYPES[xd],
                      _DTYPES[dt])
    status = load().moe_rms_norm_packed(args, _stream(stream))
    if status:
        _check(status)


def moe_quantize_rows(x, q, scales, stream=None):
    """x [T, H] (bf16, fp16 or fp32, rows may be strided) in 8 bits: q
    (float8_e4m3fn [T, H]) and scales (fp32 [T]), x standing for q * scale.  See
    the C header."""
    status = _quick_rows(x, q, scales, stream)
    if status != 1:
        if status:
            _check(status)
        return
    row = x.shape
    T, H = row
    xd, sx, sq = x.dtype, x.stride(), q.stride()
    if not (x.is_cuda and xd in _X_DTYPES and sx[1] == 1 and q.is_cuda and q.dtype == E4M3 and q.shape == row and
            sq[1] == 1 and scales.is_cuda and scales.dtype == _F32 and scales.shape == (T,) and scales.is_contiguous()):
        _rows_fault(("x", x, tuple(_X_DTYPES), row), ("q", q, (E4M3,), row), ("scales", scales, (_F32,), (T,)))
    args = _ROWS_PACK(x.data_ptr(), q.data_ptr(), scales.data_ptr(), sx[0], sq[0], _X_DTYPES[xd], T, H)
    status = load().moe_quantize_rows_packed(args, _stream(stream))
    if status:
        _check(status)


def moe_linear_8bit_workspace_size(T: int, N: int, K: int) -> int:
    return int(load().moe_linear_8bit_workspace_size(T, N, K))


def moe_linear_8bit(x, x_scales, w, w_scales, y, bias=None, act: int = MOE_ACT_NONE, residual=None, ws=None, stream=None):
    """y[T, N] = act(x[T, K] w[N, K]^T * x_scales[T] * w_scales[N] + bias[N]) +
    residual[T, N] for x and w in float8_e4m3fn with fp32 scales a row (see the C
    header).  Rows may be strided; residual may be y.  ws: a zero-filled device
    buffer of at least moe_linear_8bit_workspace_size bytes."""
    status = _quick_linear_8bit(x, x_scales, w, w_scales, y, bias, act, residual, ws, stream)
    if status != 1:
        if status:
            _check(status)
        return
    T, K = x.shape
    N = w.shape[0]
    dt = y.dtype
    sx, sw, sy = x.stride(), w.stride(), y.stride()
    if not (dt in _DTYPES and x.is_cuda and w.is_cuda and y.is_cuda and x.dtype == E4M3 and w.dtype == E4M3 and
            w.shape == (N, K) and y.shape == (T, N) and sx[1] == 1 and sw[1] == 1 and sy[1] == 1 and x_scales.is_cuda and
            w_scales.is_cuda and x_scales.dtype == _F32 and w_scales.dtype == _F32 and x_scales.shape == (T,) and
            w_scales.shape == (N,) and x_scales.is_contiguous() and w_scales.is_contiguous()):
        _rows_fault(("x", x, (E4M3,), (T, K)), ("w", w, (E4M3,), (N, K)), ("y", y, tuple(_DTYPES), (T, N)),
                    ("x_scales", x_scales, (_F32,), (T,)), ("w_scales", w_scales, (_F32,), (N,)))
    bp = rp = ldr = wp = wn = 0
    if bias is not None:
        if not (bias.is_cuda and bias.dtype == dt and bias.shape == (N,) and bias.is_contiguous()):
            _rows_fault(("bias", bias, (dt,), (N,)))
        bp = bias.data_ptr()
    if residual is not None:
        st = residual.stride()
        if not (residual.is_cuda and residual.dtype == dt and residual.shape == (T, N) and st[1] == 1):
            _rows_fault(("residual", residual, (dt,), (T, N)))
        rp, ldr = residual.data_ptr(), st[0]
    if ws is not None:
        wp, wn = _ptr(ws), ws.nbytes
    args = _LINEAR8_PACK(x.data_ptr(), x_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(), bp, rp, y.data_ptr(), wp,
                         sx[0], sw[0], ldr, sy[0], wn, T, N, K, _DTYPES[dt], act)
    status = load().moe_linear_8bit_packed(args, _stream(stream))
    if status:
        _check(status)


_SCORING_PACK = struct.Struct("@iifP3i4x").pack  # the bytes of a moe_scoring
_SCORED_PACK = struct.Struct("@PPPiifP3i4x3i4x").pack  # and of a moe_route_scored_args


def moe_route_scored(logits, k: int, ids, weights, scoring: int = MOE_SCORE_SOFTMAX, bias=None, groups: int = 1,
                     top_groups: int = 1, group_top: int = 1, renormalize: int = 1, scale: float = 1.0, stream=None):
    """The k experts of each token and their weights (ids int32 [T, k], weights
    fp32 [T, k]) from logits fp32 [T, E]: softmax or sigmoid scores, a bias (fp32
    [E]) that only the choice sees, the top_groups best of groups (by their
    group_top largest choices), weights renormalised and scaled.  See the C
    header."""
    status = _quick_route_scored(logits, k, ids, weights, scoring, bias, groups, top_groups, group_top, renormalize, scale,
                                 stream)
    if status != 1:
        if status:
            _check(status)
        return
    T, E = logits.shape
    row = (T, k)
    if not (logits.is_cuda and logits.dtype == _F32 and logits.is_contiguous() and ids.is_cuda and
            ids.dtype == torch.int32 and ids.shape == row and ids.is_contiguous() and weights.is_cuda and
            weights.dtype == _F32 and weights.shape == row and weights.is_contiguous()):
        _rows_fault(("logits", logits, (_F32,), (T, E)), ("ids", ids, (torch.int32,), row), ("weights", weights, (_F32,), row))
        raise ValueError("logits, ids and weights: expected contiguous tensors")
    bp = 0
    if bias is not None:
        if not (bias.is_cuda and bias.dtype == _F32 and bias.shape == (E,) and bias.is_contiguous()):
            _rows_fault(("bias", bias, (_F32,), (E,)))
        bp = bias.data_ptr()
    args = _SCORED_PACK(logits.data_ptr(), ids.data_ptr(), weights.data_ptr(), scoring, renormalize, scale, bp, groups,
                        top_groups, group_top, T, E, k)
    status = load().moe_route_scored_packed(args, _stream(stream))
    if status:
        _check(status)


def moe_route_tokens_scored(x, w_router, router_bias, k: int, logits, ids, weights, expert_offsets, sorted_pair,
                            pair_to_sorted, scoring: int = MOE_SCORE_SOFTMAX, bias=None, groups: int = 1,
                            top_groups: int = 1, group_top: int = 1, renormalize: int = 1, scale: float = 1.0, ws=None,
                            fresh: bool = False, stream=None):
    """moe_router_logits, moe_route_scored and moe_permute in one call (see the C
    header).  ws: a device buffer of moe_permute_workspace_size bytes, or None.
    fresh: x may be written by the kernel enqueued just before.  expert_offsets,
    sorted_pair and pair_to_sorted may be longer than E + 1 and T k."""
    T, H = x.shape
    E = w_router.shape[0]
    if x.element_size() != 2 or w_router.element_size() != 2 or w_router.shape != (E, H):
        raise ValueError(f"x, w_router: expected 16-bit [T, {H}] and [E, {H}], got {x.dtype} {tuple(x.shape)} and "
                         f"{w_router.dtype} {tuple(w_router.shape)}")
    for what, t, dt, shape in (("logits", logits, _F32, (T, E)), ("ids", ids, torch.int32, (T, k)),
                               ("weights", weights, _F32, (T, k)), ("router_bias", router_bias, _F32, (E,)),
                               ("bias", bias, _F32, (E,))):
        if t is not None and (t.dtype != dt or t.shape != shape):
            raise ValueError(f"{what}: expected {dt} {shape}, got {t.dtype} {tuple(t.shape)}")
    for what, t, n in (("expert_offsets", expert_offsets, E + 1), ("sorted_pair", sorted_pair, T * k),
                       ("pair_to_sorted", pair_to_sorted, T * k)):
        if t is not None and (t.dtype != torch.int32 or t.numel() < n):
            raise ValueError(f"{what}: expected at least {n} of torch.int32, got {t.numel()} of {t.dtype}")
    how = _SCORING_PACK(scoring, renormalize, scale, _ptr(bias) or 0, groups, top_groups, group_top)
    wp, wn = _ws(ws)
    _check(load().moe_route_tokens_scored(_ptr(x), _ptr(w_router), _ptr(router_bias), T, H, E, k, how, fresh, _ptr(logits),
                                          _ptr(ids), _ptr(weights), _ptr(expert_offsets), _ptr(sorted_pair),
                                          _ptr(pair_to_sorted), wp, wn, _stream(stream)))


# ------------------------------------------------------------------ encoder

def moe_vq2_train_codebook(W: torch.Tensor, init_idx, iters: int, stream=None):
    """The layer codebook from dense fp32 weights W [rows, K] (CUDA): k-means
    from the normalised group vectors at init_idx (128 indices).  Returns
    (codebook fp16 [128, 4], centroids fp32 [128, 4]) on the device."""
    import numpy as np
    rows, K = W.shape
    idx = np.ascontiguousarray(np.asarray(init_idx, dtype=np.int64).ravel())
    if idx.size != 128:
        raise ValueError("init_idx needs 128 indices")
    ws = torch.empty(load().moe_vq2_encoder_workspace_size(rows, K), dtype=torch.uint8, device=W.device)
    cb = torch.empty(128, 4, dtype=torch.float16, device=W.device)
    C = torch.empty(128, 4, dtype=torch.float32, device=W.device)
    _check(load().moe_vq2_train_codebook(_ptr(W), rows, K, idx.ctypes.data, iters, _ptr(cb), _ptr(C), _ptr(ws),
                                         ws.numel(), _stream(stream)))
    return cb, C


def moe_vq2_encode(W: torch.Tensor, codebook: torch.Tensor, iters: int = 3, stream=None):
    """Codes uint8 [rows, K/4] and scales fp16 [rows, K/128] (logical layout)
    of dense fp32 weights W [rows, K] (CUDA) with a fp16 codebook [128, 4]."""
    rows, K = W.shape
    ws = torch.empty(load().moe_vq2_encoder_workspace_size(rows, K), dtype=torch.uint8, device=W.device)
    codes = torch.empty(rows, K // 4, dtype=torch.uint8, device=W.device)
    scales = torch.empty(rows, K // 128, dtype=torch.float16, device=W.device)
    _check(load().moe_vq2_encode(_ptr(W), rows, K, _ptr(codebook), iters, _ptr(codes), _ptr(scales), _ptr(ws),
                                 ws.numel(), _stream(stream)))
    return codes, scales


from .layer import (GatedForward, GraphedForward, GraphedStep, MissFetchForward, MoELayer, PipelinedSteps,  # noqa: E402,F401
                    Scoring, TandemForward, host_expert, host_expert_image, upload_layer, upload_expert)
from .attention import (AttentionBatch, AttentionLayer, DecoderLayer, RMSNorm, Rows8, plan_batch,  # noqa: E402,F401
                        quantize_rows, rotation_table, upload_batch)
