"""Refusals of the grouped plans and caches and of the layer norm, before any CUDA call
(so these checks need no GPU)."""
import ctypes

import numpy as np
import pytest

from generative_recommender_ranking_gb300 import binding as bd
from generative_recommender_ranking_gb300 import build as bld

OK, INVALID, UNSUPPORTED = bd.OK, bd.ERR_INVALID_ARG, bd.ERR_UNSUPPORTED
A, B, C, D, E = (0x100000000 * i for i in range(1, 6))  # addresses that are never read


@pytest.fixture(scope="module")
def L():
    bld.build()
    return bd.lib()


def _plan(L, heads, kv, keep=-1, d=64, dtype="bf16", off=(0, 10), out=True):
    vp = ctypes.c_void_p
    off = np.asarray(off, dtype=np.int64)
    h = vp()
    L.rec_attn_plan_grouped.argtypes = [ctypes.POINTER(bd.RecAttnParams), ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_int32, vp, vp, vp, vp, vp, ctypes.POINTER(vp)]
    p = bd.make_params(heads, d, dtype=dtype)
    return L.rec_attn_plan_grouped(ctypes.byref(p), kv, keep, len(off) - 1, off.ctypes.data, A, B, C, None,
                                   ctypes.byref(h) if out else None)


@pytest.mark.parametrize("heads,kv", [(8, 0), (8, -1), (8, 3), (8, 16), (2, 4), (1, 2)])
def test_key_heads_must_divide_the_query_heads(L, heads, kv):
    assert _plan(L, heads, kv) == INVALID
    off = np.array([0, 5], dtype=np.int64)
    with pytest.raises(bd.RecAttnError) as e:
        bd.rec_attn_cache_create_grouped(bd.make_params(heads, 64), kv, off, A, B, C, D, 4, stream=0)
    assert e.value.code == INVALID


def test_plan_keeps_the_other_checks(L):
    assert _plan(L, 8, 2, keep=-2) == INVALID
    assert _plan(L, 8, 2, d=32) == UNSUPPORTED
    assert _plan(L, 8, 2, off=(0, 10, 5)) == INVALID
    assert _plan(L, 8, 2, off=(1, 10)) == INVALID
    assert _plan(L, 8, 2, out=False) == INVALID
    vp = ctypes.c_void_p
    h = vp(5)
    off = np.array([0, 1], dtype=np.int64)
    assert L.rec_attn_plan_grouped(None, 1, -1, 1, off.ctypes.data, A, B, C, None, ctypes.byref(h)) == INVALID
    assert not h.value


def _fwd(L, dtype=0, rows=4, width=64, x=A, ty=None, w=B, b=C, eps=1e-5, y=D, groups=None):
    groups = (4 if ty else 1) if groups is None else groups
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    L.rec_attn_layernorm_fwd.argtypes = [ctypes.c_int32, i64, i64, ctypes.c_int32, vp, vp, vp, vp, ctypes.c_float, vp, vp]
    return L.rec_attn_layernorm_fwd(dtype, rows, width, groups, x, ty, w, b, eps, y, None)


def _bwd(L, dtype=0, rows=4, width=64, x=A, ty=None, w=B, eps=1e-5, dy=C, dx=D, dw=E, db=E + 0x10000, groups=None):
    groups = (4 if ty else 1) if groups is None else groups
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    L.rec_attn_layernorm_bwd.argtypes = [ctypes.c_int32, i64, i64, ctypes.c_int32, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp,
                                         vp]
    return L.rec_attn_layernorm_bwd(dtype, rows, width, groups, x, ty, w, eps, dy, dx, dw, db, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_layernorm_arguments(L, call):
    assert call(L, dtype=2) == INVALID and call(L, dtype=-1) == INVALID
    assert call(L, rows=-1) == INVALID
    assert call(L, width=0) == INVALID and call(L, width=-8) == INVALID
    assert call(L, width=12) == INVALID and call(L, dtype=1, width=6) == INVALID  # rows of whole 16-byte pieces
    assert call(L, width=16392) == UNSUPPORTED
    assert call(L, rows=1 << 31) == UNSUPPORTED
    assert call(L, groups=2) == INVALID and call(L, groups=0) == INVALID
    assert call(L, groups=4) == INVALID  # by type, without the types
    assert call(L, groups=1, ty=0x700000000) == INVALID
    assert call(L, eps=-1.0) == INVALID and call(L, eps=float("nan")) == INVALID
    assert call(L, eps=float("inf")) == INVALID
    assert call(L, x=None) == INVALID and call(L, w=None) == INVALID
    assert call(L, x=A + 8) == INVALID and call(L, w=B + 4) == INVALID


def test_layernorm_overlaps(L):
    n = 4 * 64 * 2
    assert _fwd(L, y=None) == INVALID and _fwd(L, y=D + 2) == INVALID and _fwd(L, b=C + 4) == INVALID
    assert _fwd(L, y=A + 16) == INVALID and _fwd(L, y=A - n + 16) == INVALID  # partly over x
    assert _fwd(L, y=B) == INVALID and _fwd(L, y=C) == INVALID and _fwd(L, ty=D) == INVALID
    assert _bwd(L, dy=None) == INVALID and _bwd(L, dx=None) == INVALID
    assert _bwd(L, dy=C + 8) == INVALID and _bwd(L, dx=D + 8) == INVALID
    assert _bwd(L, dx=A + 16) == INVALID and _bwd(L, dx=C + 16) == INVALID
    assert _bwd(L, dx=B) == INVALID and _bwd(L, ty=D) == INVALID
    assert _bwd(L, dw=E, db=E) == INVALID and _bwd(L, dw=E + 4) == INVALID and _bwd(L, db=E + 4) == INVALID
    for over in (A, B, C, D):
        assert _bwd(L, dw=over) == INVALID and _bwd(L, db=over) == INVALID
    assert _bwd(L, ty=E) == INVALID


def test_layernorm_binding_checks_the_tensors():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(1, 64)
    ty = torch.zeros(4, dtype=torch.int8)
    bad = [
        lambda: bd.rec_attn_layernorm_fwd(x.half(), w, None, x.half(), stream=0),
        lambda: bd.rec_attn_layernorm_fwd(x.t(), w, None, x.t(), stream=0),
        lambda: bd.rec_attn_layernorm_fwd(x, w, None, x.float(), stream=0),
        lambda: bd.rec_attn_layernorm_fwd(x, w, None, x[:3], stream=0),
        lambda: bd.rec_attn_layernorm_fwd(x, w.bfloat16(), None, x, stream=0),
        lambda: bd.rec_attn_layernorm_fwd(x, w, w[:, :32], x, stream=0),
        lambda: bd.rec_attn_layernorm_fwd(x, w, None, x, types=ty, stream=0),
        lambda: bd.rec_attn_layernorm_fwd(x, w.repeat(4, 1), None, x, types=ty[:3], stream=0),
        lambda: bd.rec_attn_layernorm_fwd(x, w.repeat(4, 1), None, x, types=ty.int(), stream=0),
        lambda: bd.rec_attn_layernorm_bwd(x, w, x[:2], x, stream=0),
        lambda: bd.rec_attn_layernorm_bwd(x, w, x, x, w.repeat(4, 1), stream=0),
        lambda: bd.rec_attn_layernorm_bwd(x[0], w, x[0], x[0], stream=0),
    ]
    for call in bad:
        with pytest.raises(bd.RecAttnError) as e:
            call()
        assert e.value.code == INVALID


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_layernorm_rows_are_counted_in_32_bits(L, call):
    assert call(L, rows=(1 << 31) - 65535) == UNSUPPORTED
