"""The attention-side entry points refuse on the host what they cannot do,
before any work is enqueued (no GPU needed)."""
import ctypes

import pytest

import bit_vq_routed_gb300 as bv

P = ctypes.c_void_p
INV, UNS, WSP = bv.MOE_ERR_INVALID_ARG, bv.MOE_ERR_UNSUPPORTED, bv.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return bv.load()


def _linear(lib, **kw):
    a = dict(x=P(4096), ldx=64, w=P(4096), ldw=64, bias=None, residual=None, ldr=0, y=P(4096), ldy=32, T=4, N=32, K=64,
             dtype=0, act=0, ws=P(4096), ws_bytes=1 << 30, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.moe_linear(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV), (dict(T=-1), INV), (dict(N=-1), INV),
    (dict(K=0), INV), (dict(dtype=2), INV), (dict(act=5), INV), (dict(act=-1), INV), (dict(ldx=56), INV),
    (dict(ldw=56), INV), (dict(ldy=31), INV), (dict(residual=P(4096), ldr=31), INV), (dict(K=60), UNS),
    (dict(ldx=65), UNS), (dict(ldw=66), UNS), (dict(x=P(4104)), UNS), (dict(w=P(4098)), UNS), (dict(y=P(4097)), UNS),
    (dict(bias=P(4097)), UNS), (dict(ws=None), WSP), (dict(ws_bytes=8), WSP)])
def test_linear_refuses(lib, kw, status):
    n = bv.moe_launch_count()
    assert _linear(lib, **kw) == status
    assert b"moe_linear" in lib.moe_last_error()
    assert bv.moe_launch_count() == n


def test_empty_calls(lib):
    n = bv.moe_launch_count()
    assert _linear(lib, T=0, x=None) == 0 and _linear(lib, N=0, w=None) == 0
    assert _append(lib, T=0) == 0 and _attention(lib, T=0, q=None) == 0
    assert bv.moe_launch_count() == n


def _cache(**kw):
    c = bv._KVCache(4096, 8192)
    c.k_stride[:] = (16 * 2 * 64, 2 * 64, 64)
    c.v_stride[:] = (16 * 2 * 64, 2 * 64, 64)
    c.num_pages, c.page_size, c.kv_heads, c.head_dim, c.dtype = 8, 16, 2, 64, 0
    for k, v in kw.items():
        if k in ("k_stride", "v_stride"):
            getattr(c, k)[:] = v
        else:
            setattr(c, k, v)
    return c


def _append(lib, desc=None, **kw):
    c = _cache(**(desc or {}))
    a = dict(cache=ctypes.byref(c), k=P(4096), kt=128, kh=64, v=P(4096), vt=128, vh=64, q=P(4096), qt=256, qh=64,
             q_out=P(4096), ot=256, oh=64, q_heads=4, T=3, positions=P(4096), slots=P(4096), cos_sin=P(4096), maxp=100,
             rot=64, interleaved=0, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.moe_kv_append(*a.values())


@pytest.mark.parametrize("desc,kw,status", [
    ({}, dict(cache=None), INV), ({}, dict(k=None), INV), ({}, dict(v=None), INV), ({}, dict(slots=None), INV),
    ({}, dict(T=-1), INV), ({}, dict(positions=None), INV), ({}, dict(cos_sin=None), INV), ({}, dict(maxp=0), INV),
    ({}, dict(q_out=None), INV), ({}, dict(q_heads=0), INV), ({}, dict(rot=80), INV), ({}, dict(rot=-16), INV),
    ({}, dict(interleaved=2), INV), ({}, dict(rot=25), UNS), ({}, dict(kt=129), UNS), ({}, dict(qh=60), UNS),
    ({}, dict(k=P(4104)), UNS), ({}, dict(q=P(4100)), UNS), ({}, dict(slots=P(4100)), UNS),
    ({}, dict(positions=P(4098)), UNS), (dict(k=None), {}, INV), (dict(dtype=3), {}, INV), (dict(num_pages=0), {}, INV),
    (dict(page_size=0), {}, INV), (dict(head_dim=60), {}, UNS), (dict(head_dim=264), {}, UNS),
    (dict(k_stride=(2048, 128, 60)), {}, UNS), (dict(v=8200), {}, UNS)])
def test_append_refuses(lib, desc, kw, status):
    n = bv.moe_launch_count()
    assert _append(lib, desc, **kw) == status
    assert b"moe_kv_append" in lib.moe_last_error()
    assert bv.moe_launch_count() == n


def _attention(lib, desc=None, **kw):
    c = _cache(**(desc or {}))
    a = dict(cache=ctypes.byref(c), q=P(4096), qt=256, qh=64, q_heads=4, T=3, cu_q=P(4096), B=2, prefix_pages=P(4096),
             prefix_len=40, page_table=P(4096), table_stride=4, max_pages=4, seq_lens=P(4096), scale=0.125, out=P(4096),
             ot=256, oh=64, lse=None, ws=P(4096), ws_bytes=1 << 40, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.moe_prefix_attention(*a.values())


@pytest.mark.parametrize("desc,kw,status", [
    ({}, dict(cache=None), INV), ({}, dict(q=None), INV), ({}, dict(out=None), INV), ({}, dict(cu_q=None), INV),
    ({}, dict(seq_lens=None), INV), ({}, dict(prefix_pages=None), INV), ({}, dict(page_table=None), INV),
    ({}, dict(table_stride=3), INV), ({}, dict(T=-1), INV), ({}, dict(B=0), INV), ({}, dict(prefix_len=-1), INV),
    ({}, dict(max_pages=-1), INV), ({}, dict(scale=0.0), INV), ({}, dict(scale=-1.0), INV),
    ({}, dict(scale=float("nan")), INV), ({}, dict(scale=float("inf")), INV), ({}, dict(q_heads=3), INV),
    ({}, dict(q_heads=0), INV), ({}, dict(q_heads=258), UNS), ({}, dict(qt=257), UNS), ({}, dict(oh=68), UNS),
    ({}, dict(q=P(4104)), UNS), ({}, dict(out=P(4098)), UNS), ({}, dict(ws=None), WSP), ({}, dict(ws_bytes=16), WSP),
    (dict(v=None), {}, INV), (dict(dtype=-1), {}, INV), (dict(kv_heads=0), {}, INV), (dict(head_dim=136), {}, UNS),
    (dict(head_dim=60), {}, UNS), (dict(page_size=24), {}, UNS), (dict(page_size=4), {}, UNS),
    (dict(page_size=2048), {}, UNS), (dict(v_stride=(2048, 124, 64)), {}, UNS), (dict(k=4104), {}, UNS)])
def test_attention_refuses(lib, desc, kw, status):
    n = bv.moe_launch_count()
    assert _attention(lib, desc, **kw) == status
    assert b"moe_prefix_attention" in lib.moe_last_error()
    assert bv.moe_launch_count() == n


def test_workspace_sizes(lib):
    assert bv.moe_linear_workspace_size(1, 4096, 4096) >= 16
    assert bv.moe_linear_workspace_size(-1, 1, 8) == 0 and bv.moe_linear_workspace_size(1, 1, 0) == 0
    assert bv.moe_prefix_attention_workspace_size(1, 8, 2, 128) >= 16
    assert bv.moe_prefix_attention_workspace_size(1, 8, 0, 128) == 0


def test_packed_append_takes_the_header_struct(lib):
    # the bytes that the binding packs, read back through the same call's checks
    def call(**kw):
        a = dict(kc=4096, vc=4096, ks=(2048, 128, 64), vs=(2048, 128, 64), size=(8, 16, 2, 64, 0), k=4096, v=4096, q=4096,
                 q_out=4096, s=(128, 64, 128, 64, 256, 64, 256, 64), pos=4096, slots=4096, table=4096,
                 n=(4, 3, 100, 64, 0))
        a.update(kw)
        b = bv._APPEND_PACK(a["kc"], a["vc"], *a["ks"], *a["vs"], *a["size"], a["k"], a["v"], a["q"], a["q_out"], *a["s"],
                            a["pos"], a["slots"], a["table"], *a["n"])
        return lib.moe_kv_append_packed(b, None)

    n = bv.moe_launch_count()
    assert lib.moe_kv_append_packed(None, None) == INV
    for kw, status, text in [
            (dict(k=0), INV, b"null"), (dict(table=0), INV, b"cos_sin"), (dict(n=(4, 3, 100, 64, 2)), INV, b"interleaved=2"),
            (dict(n=(4, -1, 100, 64, 0)), INV, b"T=-1"), (dict(n=(4, 3, 100, 25, 0)), UNS, b"rot_dim=25"),
            (dict(size=(8, 16, 2, 60, 0)), UNS, b"head_dim=60"), (dict(size=(8, 16, 2, 64, 3)), INV, b"dtype 3"),
            (dict(s=(128, 64, 128, 64, 256, 64, 256, 60)), UNS, b"strides"), (dict(slots=4100), UNS, b"slots")]:
        assert call(**kw) == status, kw
        assert text in lib.moe_last_error(), kw
    assert call(n=(4, 0, 100, 64, 0)) == bv.MOE_OK  # T = 0 enqueues nothing
    assert bv.moe_launch_count() == n
