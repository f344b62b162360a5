"""Host-side checks of the cache, bounds and selection entry points: every
refusal comes before any device work."""
import ctypes
import types

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


def test_scaled_attention_refusals(lib):  # noqa: F811
    """The entry points with scales: 8-bit K/V only, scales required, the other
    checks as for the entry points without; those refuse 8-bit K/V."""
    from block_sparse_paged_csr_gb300 import _native

    n = _names()
    cu = np.array([0, 1, 2, 3, 4], np.int64)
    pcu = cu.ctypes.data_as(ctypes.c_void_p)

    def index(**kw):
        a = dict(hkv=2, pages_per_block=4, block_size=64, page_size=16, tq=4, topk=2, batch=4, msb=2)
        a.update(kw)
        return _native.SaIndex(**a)

    def fwd(idx=None, qt=0, kv=2, ks=P, vs=P, hq=4, hkv=2, d=128, bs=64, ps=16, causal=0, path=0,
            pdt=0, q=P):
        idx = index() if idx is None else idx
        return lib.sa_forward_scaled(q, qt, P, P, ks, vs, 16, kv, ctypes.byref(idx), P, P, None, hq,
                                     hkv, d, bs, ps, 0.1, causal, pdt, P, P, P, path, None)

    assert fwd(hq=3) == n["HEAD_COUNT"]
    assert fwd(bs=24) == n["BLOCK_PAGE"]
    assert fwd(bs=32) == n["SHAPE"]
    assert fwd(kv=0) == n["INVALID_ARGUMENT"]
    assert fwd(kv=1) == n["INVALID_ARGUMENT"]
    assert fwd(kv=4) == n["INVALID_ARGUMENT"]
    assert fwd(qt=2) == n["INVALID_ARGUMENT"]
    assert fwd(pdt=2) == n["INVALID_ARGUMENT"]
    assert fwd(causal=3) == n["INVALID_ARGUMENT"]
    assert fwd(path=4) == n["UNSUPPORTED"]
    assert fwd(d=40) == n["UNSUPPORTED"]
    assert fwd(ks=None) == n["INVALID_ARGUMENT"]
    assert fwd(vs=None) == n["INVALID_ARGUMENT"]
    assert fwd(q=ODD) == n["INVALID_ARGUMENT"]

    def both(kv=2, ks=P, vs=P, path=0, hq=4, q=P, ws=P, cu_host=pcu):
        idx = index(workspace=4096, workspace_bytes=1 << 20, inv=4096, totals=4096)
        if ws is None:
            idx.workspace = None
        return lib.sa_forward_combine_scaled(q, 0, P, P, ks, vs, 16, kv, ctypes.byref(idx), P,
                                             cu_host, P, None, P, hq, 128, 64, 16, 0.1, 1, 0, 0, P, P,
                                             P, P, P, path, None)

    assert both(kv=1) == n["INVALID_ARGUMENT"]
    assert both(hq=3) == n["HEAD_COUNT"]
    assert both(ks=None) == n["INVALID_ARGUMENT"]
    assert both(q=ODD) == n["INVALID_ARGUMENT"]
    assert both(ws=None) == n["INVALID_ARGUMENT"]      # the fused path's counters
    assert both(hq=34, path=4) == n["UNSUPPORTED"]     # 17 lanes

    def att(kv=3, hq=4, d=128, bs=64, causal=1, path=0, sel=None):
        idx = _native.SaIndex()
        return lib.sa_attention_scaled(P, 0, P, P, P, P, 16, kv, sel, 4, 2, pcu, P, 4, None, P, 8, hq,
                                       2, d, bs, 16, 0.1, causal, 0, ctypes.byref(idx), 0, P, P, P, P,
                                       P, path, None)

    assert att(kv=0) == n["INVALID_ARGUMENT"]
    assert att(hq=5) == n["HEAD_COUNT"]
    assert att(bs=40) == n["BLOCK_PAGE"]
    assert att(d=24) == n["UNSUPPORTED"]
    assert att(causal=7) == n["INVALID_ARGUMENT"]
    assert att(path=4, causal=2) == n["UNSUPPORTED"]
    assert att() == n["INVALID_ARGUMENT"]              # no selection, no index arrays
    # without scales: the 8-bit types are refused as before
    idx = index()
    assert lib.sa_forward(P, P, P, 16, 2, ctypes.byref(idx), P, P, None, 4, 2, 128, 64, 16, 0.1, 0,
                          P, P, P, 0, None) == n["INVALID_ARGUMENT"]


def test_scaled_kernel_choice():
    import block_sparse_paged_csr_gb300 as sa

    one = np.array([0, 1, 1, 2, 3], np.int64)
    many = np.array([0, 40, 80], np.int64)
    name = sa.sa_attention_kernel_name
    for kind in ("e4m3", "int8"):
        assert name(one, 1000, 8, 32, 128, 64, 16, kind) == "fused_dec_kernel"
        assert name(one, 1000, 2, 32, 128, 64, 16, kind) == "fused_dec_kernel"
        assert name(one, 1000, 1, 32, 128, 64, 16, kind) == "forward_cc_kernel"   # 32 lanes
        assert name(one, 1000, 8, 32, 128, 64, 8, kind) == "forward_cc_kernel"    # pages of 8
        assert name(one, 1000, 8, 32, 64, 64, 16, kind) == "forward_cc_kernel"
        assert name(one, 1000, 8, 32, 128, 64, 16, kind, causal=2) == "forward_cc_kernel"
        assert name(many, 1000, 8, 64, 128, 128, 64, kind) == "forward_tc_kernel"
        assert name(many, 1000, 8, 64, 64, 128, 64, kind) == "forward_cc_kernel"
        assert name(many, 1000, 8, 64, 72, 128, 64, kind) is None
        assert sa.sa_forward_kernel_name(80, 2, 8, 64, 128, 128, 64, kind,
                                         sa.PATH_TENSOR_CORE) == "forward_tc_kernel"
        assert sa.sa_forward_kernel_name(80, 2, 8, 64, 128, 128, 64, kind,
                                         sa.PATH_CUDA_CORE) == "forward_cc_kernel"


def test_host_pointers():
    """Host prefix lengths reach the library by the address of their data,
    writable or not, whatever they come as."""
    import torch

    import block_sparse_paged_csr_gb300 as sa

    a = np.arange(5, dtype=np.int64)
    p = sa._host_ptr(a)
    assert ctypes.addressof(p) == a.ctypes.data
    a.flags.writeable = False
    assert sa._host_ptr(a) == a.ctypes.data
    for x in ([0, 2, 5], np.array([0, 2, 5], np.int32), torch.tensor([0, 2, 5])):
        h = sa._host_i64(x)
        assert h.dtype == np.int64 and h.flags.c_contiguous and h.tolist() == [0, 2, 5]


@pytest.mark.parametrize("shape", [(4, 2, 32, 128), (4, 1, 16, 128), (4, 2, 16, 64), (4, 4, 8, 128)])
def test_pool_of_other_sizes(shape):
    """An 8-bit pool whose shape is not what the call's sizes say is refused
    before any pointer is taken: its scales would be read past their end."""
    import torch

    import block_sparse_paged_csr_gb300 as sa

    codes = torch.zeros(shape, dtype=torch.int8)
    scales = torch.ones(shape[:2])
    q = torch.zeros((1, 4, 128))
    with pytest.raises(ValueError, match="k_pages must be"):
        sa._scaled(q, codes, codes, scales, scales, 2, 16, 128)
    i32 = torch.zeros((1, 8), dtype=torch.int32)
    sel = torch.zeros((1, 2, 1), dtype=torch.int32)
    with pytest.raises(ValueError, match="k_pages must be"):
        sa.sa_attention(q, codes, codes, sel, [0, 1], None, None, i32, 4, 2, 128, 64, 16, 0.1, True,
                        k_scales=scales, v_scales=scales)
    with pytest.raises(ValueError, match="k_pages must be"):
        sa.sa_forward(q, codes, codes, None, i32, None, None, 4, 2, 128, 64, 16, 0.1, True,
                      k_scales=scales, v_scales=scales)
    index = sa._native.SaIndex(hkv=2, tq=1)
    with pytest.raises(ValueError, match="k_pages must be"):
        sa.sa_forward_combine(q, codes, codes, types.SimpleNamespace(c=index), sel, [0, 1], None, None,
                              i32, 4, 128, 64, 16, 0.1, True, k_scales=scales, v_scales=scales)


def test_kernel_names_are_kernels():
    """What the name queries answer is the name of a kernel in the file that
    serves the cache type (a profiling script filters by it)."""
    import os
    import re

    import block_sparse_paged_csr_gb300 as sa

    csrc = os.path.join(os.path.dirname(sa.__file__), "csrc")

    def kernels(file):
        with open(os.path.join(csrc, file)) as f:
            return set(re.findall(r"__global__[^;{]*?\b(\w+)\(const|__global__[^;{]*?\b(\w+)\(ForwardArgs",
                                  f.read()))

    one, many = np.arange(5, dtype=np.int64), np.array([0, 40, 80], np.int64)
    for kind in ("f32", "bf16", "e4m3", "int8"):
        eight = kind in ("e4m3", "int8")
        for cu, d, path, file in (
                (one, 128, sa.PATH_AUTO, "fused_dec_q8.cu" if eight else "fused_dec.cu"),
                (many, 128, sa.PATH_AUTO, "forward_tc.cu"),
                (many, 64, sa.PATH_AUTO, "forward_cc.cu")):
            name = sa.sa_attention_kernel_name(cu, 1000, 8, 32, d, 64, 16, kind, path=path)
            assert name in {n for pair in kernels(file) for n in pair}, (kind, name, file)


def test_index_of_a_smaller_problem():
    """An index handed in has to hold one over the call's sizes."""
    import block_sparse_paged_csr_gb300 as sa

    small = types.SimpleNamespace(sizes=sa.sa_index_query_sizes(4, 2, 3, 4, 16, 64, 16))
    sa._check_index(small, 4, 2, 3, 4, 16, 64, 16)
    sa._check_index(small, 2, 2, 3, 2, 16, 64, 16)          # larger than needed
    sa._check_index(small, 4, 2, 3, 4, 16, 24, 16)          # the library refuses these sizes
    for sizes in ((5, 2, 3, 4, 16), (4, 4, 3, 4, 16), (4, 2, 4, 4, 16), (4, 2, 3, 5, 16), (4, 2, 3, 4, 20)):
        with pytest.raises(ValueError, match="smaller problem"):
            sa._check_index(small, *sizes, 64, 16)
