"""Host-side checks of the cache, bounds and selection entry points: every
refusal comes before any device work."""
import ctypes

import numpy as np
import pytest

from test_library_cpu import lib  # noqa: F401  (fixture)


def _names():
    from block_sparse_paged_csr_gb300 import _native

    return {v: k for k, v in _native.STATUS_NAMES.items()}


P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4096 + 8)


def _store(lib, **kw):  # noqa: F811
    a = dict(k=P, v=P, src=0, strides=(64, 32, 64, 32), kp=P, vp=P, ks=P, vs=P, pages=8, kv=2,
             bt=P, max_pages=4, cu=np.array([0, 4], np.int64), cud=P, batch=1, tq=4, used=P, hkv=2,
             d=32, ps=16)
    a.update(kw)
    cu = a["cu"]
    return lib.sa_store_kv(a["k"], a["v"], a["src"], *a["strides"], a["kp"], a["vp"], a["ks"],
                           a["vs"], a["pages"], a["kv"], a["bt"], a["max_pages"],
                           None if cu is None else cu.ctypes.data_as(ctypes.c_void_p), a["cud"],
                           a["batch"], a["tq"], a["used"], a["hkv"], a["d"], a["ps"], None, None)


def test_store_refusals(lib):  # noqa: F811
    n = _names()
    assert _store(lib, hkv=0) == n["HEAD_COUNT"]
    assert _store(lib, d=0) == n["BLOCK_PAGE"]
    assert _store(lib, ps=0) == n["BLOCK_PAGE"]
    assert _store(lib, cu=None) == n["CU_SEQLENS"]
    assert _store(lib, cu=np.array([1, 4], np.int64)) == n["CU_SEQLENS"]
    assert _store(lib, cu=np.array([0, 3, 2], np.int64), batch=2) == n["CU_SEQLENS"]
    assert _store(lib, tq=5) == n["SHAPE"]
    assert _store(lib, pages=-1) == n["SHAPE"]
    assert _store(lib, src=2) == n["INVALID_ARGUMENT"]
    assert _store(lib, kv=4) == n["INVALID_ARGUMENT"]
    assert _store(lib, kv=-1) == n["INVALID_ARGUMENT"]
    assert _store(lib, d=24) == n["UNSUPPORTED"]          # 8-bit pages: multiples of 16
    assert _store(lib, d=12, kv=0) == n["UNSUPPORTED"]
    assert _store(lib, d=272) == n["UNSUPPORTED"]
    for name in ("k", "v", "kp", "vp", "bt", "cud", "used", "ks", "vs"):
        assert _store(lib, **{name: None}) == n["INVALID_ARGUMENT"], name
    for name in ("k", "v", "kp", "vp"):
        assert _store(lib, **{name: ODD}) == n["INVALID_ARGUMENT"], name
    assert _store(lib, strides=(66, 32, 64, 32)) == n["INVALID_ARGUMENT"]
    assert _store(lib, strides=(64, 32, 64, 34)) == n["INVALID_ARGUMENT"]
    assert _store(lib, src=1, strides=(64, 36, 64, 32)) == n["INVALID_ARGUMENT"]
    # nothing to store: done, whatever the pointers
    assert _store(lib, cu=np.array([0, 0], np.int64), tq=0, k=None, kp=None) == n["OK"]


def _bounds(lib, **kw):  # noqa: F811
    a = dict(kp=P, ks=P, pages=8, kv=3, bt=P, max_pages=4, cu=np.array([0, 4], np.int64), cud=P,
             batch=1, tq=4, used=P, hkv=2, d=32, bs=32, ps=16, rows=P, msb=2, n=4, out=P)
    a.update(kw)
    return lib.sa_block_bounds(a["kp"], a["ks"], a["pages"], a["kv"], a["bt"], a["max_pages"],
                               a["cu"].ctypes.data_as(ctypes.c_void_p), a["cud"], a["batch"],
                               a["tq"], a["used"], a["hkv"], a["d"], a["bs"], a["ps"], a["rows"],
                               a["msb"], a["n"], a["out"], None, None)


def test_bounds_refusals(lib):  # noqa: F811
    n = _names()
    assert _bounds(lib, hkv=0) == n["HEAD_COUNT"]
    assert _bounds(lib, bs=24) == n["BLOCK_PAGE"]
    assert _bounds(lib, bs=0) == n["BLOCK_PAGE"]
    assert _bounds(lib, cu=np.array([2, 4], np.int64)) == n["CU_SEQLENS"]
    assert _bounds(lib, tq=3) == n["SHAPE"]
    assert _bounds(lib, n=-1) == n["SHAPE"]
    assert _bounds(lib, kv=5) == n["INVALID_ARGUMENT"]
    assert _bounds(lib, d=40) == n["UNSUPPORTED"]
    for name in ("kp", "ks", "bt", "cud", "used", "rows", "out"):
        assert _bounds(lib, **{name: None}) == n["INVALID_ARGUMENT"], name
    assert _bounds(lib, kp=ODD) == n["INVALID_ARGUMENT"]
    assert _bounds(lib, cu=np.array([0, 0], np.int64), tq=0) == n["OK"]


def _select(lib, **kw):  # noqa: F811
    a = dict(q=P, qt=0, tq=4, hq=4, hkv=2, d=32, bounds=P, n=4, rows=P, msb=8,
             cu=np.array([0, 4], np.int64), cud=P, batch=1, used=P, bs=32, topk=4, causal=1, sink=0,
             local=0, sel=P, ws=P, ws_bytes=1 << 20)
    a.update(kw)
    cu = a["cu"]
    return lib.sa_select_blocks(a["q"], a["qt"], a["tq"], a["hq"], a["hkv"], a["d"], a["bounds"],
                                a["n"], a["rows"], a["msb"],
                                None if cu is None else cu.ctypes.data_as(ctypes.c_void_p),
                                a["cud"], a["batch"], a["used"], a["bs"], a["topk"], a["causal"],
                                a["sink"], a["local"], a["sel"], a["ws"], a["ws_bytes"], None, None)


def test_select_refusals(lib):  # noqa: F811
    n = _names()
    assert _select(lib, hq=3) == n["HEAD_COUNT"]
    assert _select(lib, hkv=0) == n["HEAD_COUNT"]
    assert _select(lib, d=0) == n["BLOCK_PAGE"]
    assert _select(lib, bs=0) == n["BLOCK_PAGE"]
    assert _select(lib, tq=0) == n["EMPTY"]
    assert _select(lib, topk=0) == n["EMPTY"]
    assert _select(lib, msb=-1) == n["SHAPE"]
    assert _select(lib, cu=None) == n["CU_SEQLENS"]
    assert _select(lib, cu=np.array([0, 5], np.int64)) == n["SHAPE"]
    assert _select(lib, qt=2) == n["INVALID_ARGUMENT"]
    assert _select(lib, causal=3) == n["INVALID_ARGUMENT"]
    assert _select(lib, sink=-1) == n["INVALID_ARGUMENT"]
    assert _select(lib, sink=3, local=2) == n["INVALID_ARGUMENT"]
    assert _select(lib, d=36) == n["UNSUPPORTED"]
    assert _select(lib, d=264) == n["UNSUPPORTED"]
    assert _select(lib, msb=16385) == n["UNSUPPORTED"]
    for name in ("q", "bounds", "rows", "cud", "used", "sel", "ws"):
        assert _select(lib, **{name: None}) == n["INVALID_ARGUMENT"], name
    assert _select(lib, q=ODD) == n["INVALID_ARGUMENT"]
    assert _select(lib, ws=ODD) == n["INVALID_ARGUMENT"]
    assert _select(lib, ws_bytes=16) == n["INVALID_ARGUMENT"]


def test_select_workspace_size(lib):  # noqa: F811
    n = _names()
    b = ctypes.c_size_t(0)
    assert lib.sa_select_workspace_size(64, 64, 8, 128, 512, ctypes.byref(b)) == 0
    assert 64 * 8 * 512 * 4 <= b.value < 4 << 20
    # large problems run in parts: the scratch stays bounded
    assert lib.sa_select_workspace_size(1 << 20, 64, 8, 128, 16384, ctypes.byref(b)) == 0
    assert b.value < 300 << 20
    assert lib.sa_select_workspace_size(64, 64, 8, 128, 512, None) == n["INVALID_ARGUMENT"]
    assert lib.sa_select_workspace_size(64, 64, 0, 128, 512, ctypes.byref(b)) == n["HEAD_COUNT"]
    assert lib.sa_select_workspace_size(64, 64, 8, 128, 16385, ctypes.byref(b)) == n["UNSUPPORTED"]
    assert lib.sa_select_workspace_size(64, 0, 8, 128, 512, ctypes.byref(b)) == n["CU_SEQLENS"]


def test_binding_refusals():
    """Argument checks of the Python side that need no device."""
    import torch

    import block_sparse_paged_csr_gb300 as sa

    x = torch.zeros((2, 2, 32))
    with pytest.raises(TypeError):
        sa._cache_dtype(torch.zeros((1, 2, 16, 32), dtype=torch.float16), "k_pages")
    with pytest.raises(ValueError):
        sa._cache_dtype(x, "k_pages")
    codes = torch.zeros((3, 2, 16, 32), dtype=torch.int8)
    with pytest.raises(ValueError):
        sa._scales(None, codes, "k_scales")
    with pytest.raises(ValueError):
        sa._scales(torch.zeros((3, 2)), codes.float(), "k_scales")
    with pytest.raises(TypeError):
        sa.sa_select_blocks(x.half(), None, None, [0, 2], None, None, 16, 2, True)
