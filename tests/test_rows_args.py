"""The norm, the 8-bit rows and products and the choice by score refuse on the
host what they cannot do, before any work is enqueued (no GPU needed)."""
import ctypes
import struct

import pytest

import bit_vq_routed_gb300 as bv

P = ctypes.c_void_p
INV, UNS, WSP = bv.MOE_ERR_INVALID_ARG, bv.MOE_ERR_UNSUPPORTED, bv.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return bv.load()


def _refused(lib, call, name, kw, status):
    n = bv.moe_launch_count()
    assert call(lib, **kw) == status
    assert name in lib.moe_last_error()
    assert bv.moe_launch_count() == n


def _norm(lib, **kw):
    a = dict(x=P(4096), ldx=64, x_dtype=0, residual=P(8192), ldr=64, h=P(8192), ldh=64, weight=P(512), eps=1e-6, y=P(4096),
             ldy=64, q=P(4096), ldq=64, scales=P(64), T=4, H=64, dtype=0, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.moe_rms_norm(*a.values())


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(H=0), INV), (dict(dtype=2), INV), (dict(dtype=-1), INV), (dict(x_dtype=1), INV),
    (dict(x_dtype=3), INV), (dict(eps=-1e-6), INV), (dict(eps=NAN), INV), (dict(eps=INF), INV), (dict(x=None), INV),
    (dict(y=None, q=None, scales=None), INV), (dict(q=None), INV), (dict(scales=None), INV), (dict(residual=None), INV),
    (dict(ldx=63), INV), (dict(ldr=63), INV), (dict(ldh=63), INV), (dict(ldy=63), INV), (dict(ldq=63), INV),
    (dict(H=16385, ldx=20000, ldr=20000, ldh=20000, ldy=20000, ldq=20000), UNS), (dict(x=P(4097)), UNS),
    (dict(x=P(4098), x_dtype=2), UNS), (dict(weight=P(513)), UNS), (dict(scales=P(66)), UNS), (dict(h=P(8193)), UNS),
    (dict(y=P(8193)), UNS), (dict(residual=P(8193)), UNS)])
def test_norm_refuses(lib, kw, status):
    _refused(lib, _norm, b"moe_rms_norm", kw, status)


def _quantize(lib, **kw):
    a = dict(x=P(4096), ldx=64, x_dtype=0, q=P(4096), ldq=64, scales=P(64), T=4, H=64, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.moe_quantize_rows(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(H=-1), INV), (dict(x_dtype=3), INV), (dict(x=None), INV), (dict(q=None), INV),
    (dict(scales=None), INV), (dict(ldx=63), INV), (dict(ldq=63), INV),
    (dict(H=2 ** 31 - 1, ldx=2 ** 31, ldq=2 ** 31), UNS), (dict(x=P(4097)), UNS), (dict(x=P(4098), x_dtype=2), UNS), (dict(scales=P(65)), UNS)])
def test_quantize_refuses(lib, kw, status):
    _refused(lib, _quantize, b"moe_quantize_rows", kw, status)


def _linear(lib, **kw):
    a = dict(x=P(4096), ldx=64, x_scales=P(64), w=P(4096), ldw=64, w_scales=P(64), bias=None, residual=None, ldr=0, y=P(4096),
             ldy=32, T=4, N=32, K=64, dtype=0, act=0, ws=P(4096), ws_bytes=1 << 30, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.moe_linear_8bit(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV), (dict(x_scales=None), INV), (dict(w_scales=None), INV),
    (dict(T=-1), INV), (dict(N=-1), INV), (dict(K=0), INV), (dict(dtype=2), INV), (dict(act=5), INV), (dict(act=-1), INV),
    (dict(ldx=48), INV), (dict(ldw=48), INV), (dict(ldy=31), INV), (dict(residual=P(4096), ldr=31), INV), (dict(K=56), UNS),
    (dict(ldx=72), UNS), (dict(ldw=65), UNS), (dict(x=P(4104)), UNS), (dict(w=P(4098)), UNS), (dict(y=P(4097)), UNS),
    (dict(bias=P(4097)), UNS), (dict(x_scales=P(66)), UNS), (dict(w_scales=P(66)), UNS), (dict(ws=None), WSP),
    (dict(ws_bytes=8), WSP), (dict(ws=P(4100)), UNS)])
def test_linear_8bit_refuses(lib, kw, status):
    _refused(lib, _linear, b"moe_linear_8bit", kw, status)


def _route(lib, null=False, **kw):
    a = dict(logits=P(4096), T=4, E=64, k=4, ids=P(4096), weights=P(4096))
    s = dict(scoring=1, renormalize=1, scale=1.0, bias=0, groups=4, top_groups=2, group_top=2)
    for n, v in kw.items():
        (a if n in a else s)[n] = v
    assert len(a) == 6 and len(s) == 7
    how = None if null else struct.pack("@iifP3i4x", *s.values())
    return lib.moe_route_scored(a["logits"], a["T"], a["E"], a["k"], how, a["ids"], a["weights"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(null=True), INV), (dict(T=-1), INV), (dict(E=0), INV), (dict(E=1028), UNS), (dict(k=0), INV), (dict(k=33), INV),
    (dict(top_groups=1, k=17), INV), (dict(scoring=2), INV), (dict(scoring=-1), INV), (dict(renormalize=2), INV),
    (dict(scale=NAN), INV), (dict(scale=INF), INV), (dict(groups=0), INV), (dict(groups=3), INV), (dict(groups=128), INV),
    (dict(groups=64, group_top=1), UNS), (dict(top_groups=0), INV), (dict(top_groups=5), INV), (dict(group_top=0), INV),
    (dict(group_top=3), INV), (dict(groups=32, E=32, group_top=2), INV), (dict(logits=None), INV), (dict(ids=None), INV),
    (dict(weights=None), INV), (dict(logits=P(4098)), UNS), (dict(bias=4098), UNS), (dict(ids=P(4098)), UNS),
    (dict(weights=P(4098)), UNS)])
def test_route_scored_refuses(lib, kw, status):
    _refused(lib, _route, b"moe_route_scored", kw, status)


def test_empty_calls(lib):
    n = bv.moe_launch_count()
    assert _norm(lib, T=0, x=None) == 0 and _quantize(lib, T=0, x=None) == 0
    assert _linear(lib, T=0, x=None) == 0 and _linear(lib, N=0, w=None) == 0 and _route(lib, T=0, logits=None) == 0
    assert bv.moe_launch_count() == n


def test_python_calls_refuse_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    bf, f8 = torch.zeros(2, 16, dtype=torch.bfloat16), torch.zeros(2, 16).to(torch.float8_e4m3fn)
    f = torch.zeros(2)
    for call in (lambda: bv.moe_rms_norm(bf, None, 1e-6, y=bf), lambda: bv.moe_quantize_rows(bf, f8, f),
                 lambda: bv.moe_linear_8bit(f8, f, f8, f, torch.zeros(2, 2, dtype=torch.bfloat16)),
                 lambda: bv.moe_route_scored(torch.zeros(2, 16), 2, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_packed_calls_read_their_structs(lib):
    """The calls with their arguments in a struct refuse what the others do, and say
    what they read at the struct's end."""
    norm = struct.Struct("@7P5qf4i4x").pack
    n = bv.moe_launch_count()
    assert lib.moe_rms_norm_packed(None, None) == INV and lib.moe_linear_8bit_packed(None, None) == INV
    assert lib.moe_rms_norm_packed(norm(*([4096] * 7), *([64] * 5), 1e-6, -3, 77, 0, 0), None) == INV
    assert b"T=-3" in lib.moe_last_error() and b"H=77" in lib.moe_last_error()
    assert lib.moe_rms_norm_packed(norm(*([4096] * 7), *([64] * 5), 1e-6, 4, 64, 2, 5), None) == INV
    assert b"dtype 5" in lib.moe_last_error()
    assert lib.moe_rms_norm_packed(norm(4096, 0, 4096, 0, 0, 0, 0, *([64] * 5), 1e-6, 4, 64, 0, 0), None) == INV
    assert b"y and q" in lib.moe_last_error()
    lin = struct.Struct("@8P4qN5i4x").pack
    assert lib.moe_linear_8bit_packed(lin(*([4096] * 8), 64, 64, 32, 32, 256, -4, 32, 64, 0, 0), None) == INV
    assert b"T=-4 N=32" in lib.moe_last_error()
    assert lib.moe_linear_8bit_packed(lin(*([4096] * 8), 64, 64, 32, 32, 256, 4, 32, 64, 0, 9), None) == INV
    assert b"activation 9" in lib.moe_last_error()
    assert lib.moe_linear_8bit_packed(lin(*([4096] * 8), 64, 64, 32, 32, 8, 4, 32, 64, 0, 0), None) == WSP
    assert lib.moe_linear_8bit_packed(lin(*([4096] * 7), 0, 64, 64, 32, 32, 256, 4, 32, 64, 0, 0), None) == WSP
    scored = struct.Struct("@PPPiifP3i4x3i4x").pack
    assert lib.moe_route_scored_packed(None, None) == INV
    assert lib.moe_route_scored_packed(scored(4096, 4096, 4096, 1, 1, 1.0, 0, 4, 2, 2, 4, 64, 99), None) == INV
    assert b"k=99" in lib.moe_last_error() and b"the 32 experts" in lib.moe_last_error()
    assert lib.moe_route_scored_packed(scored(4096, 4096, 4096, 1, 1, 1.0, 4098, 4, 2, 2, 4, 64, 4), None) == UNS
    rows = struct.Struct("@PPPqq3i4x").pack
    assert lib.moe_quantize_rows_packed(None, None) == INV
    assert lib.moe_quantize_rows_packed(rows(4096, 4096, 4096, 64, 64, 0, -2, 55), None) == INV
    assert b"T=-2" in lib.moe_last_error() and b"H=55" in lib.moe_last_error()
    assert lib.moe_quantize_rows_packed(rows(4096, 4096, 4096, 64, 63, 2, 2, 64), None) == INV
    assert bv.moe_launch_count() == n


def _tokens(lib, **kw):
    a = dict(x=P(4096), w=P(4096), rb=None, T=4, H=256, E=64, k=4, how=None, fresh=0, logits=P(4096), ids=P(4096),
             weights=P(4096), offsets=P(4096), sp=P(4096), ps=P(4096), ws=None, ws_bytes=0, stream=None)
    s = dict(scoring=1, renormalize=1, scale=1.0, bias=0, groups=4, top_groups=2, group_top=2)
    for n, v in kw.items():
        (a if n in a else s)[n] = v
    a["how"] = struct.pack("@iifP3i4x", *s.values())
    return lib.moe_route_tokens_scored(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(logits=None), INV), (dict(ids=None), INV), (dict(weights=None), INV),
    (dict(offsets=None), INV), (dict(sp=None), INV), (dict(ps=None), INV), (dict(H=0), INV), (dict(H=128), UNS),
    (dict(T=-1), INV), (dict(E=1028), UNS), (dict(k=0), INV), (dict(groups=3), INV), (dict(T=1 << 23), UNS), (dict(x=P(4104)), UNS),
    (dict(w=P(4104)), UNS), (dict(logits=P(4104)), UNS), (dict(rb=P(4104)), UNS), (dict(bias=4098), UNS)])
def test_route_tokens_scored_refuses(lib, kw, status):
    _refused(lib, _tokens, b"moe_route_tokens_scored", kw, status)
