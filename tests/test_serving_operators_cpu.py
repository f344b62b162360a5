"""Host-side checks of sa_norm_rope, sa_load_kv and sa_decode_attention: the
documented status codes in the documented order, before any device work."""
import ctypes
import os

import numpy as np
import pytest

F32, BF16, E4M3, INT8 = 0, 1, 2, 3
P = 1 << 20                  # an aligned address that is never read: the checks come first


@pytest.fixture(scope="module")
def lib():
    from block_sparse_paged_csr_gb300 import _native

    if not os.path.exists(_native.LIB_PATH):
        from block_sparse_paged_csr_gb300 import build

        build.build_library()
    return _native.load()


CU = np.array([0, 3, 5], np.int64)


def host(cu):
    return None if cu is None else cu.ctypes.data


def rope(lib, q=P, k=P, src=F32, qw=P, kw=P, wt=F32, eps=1e-6, freq=P, rot=64, axes=None, pos=P,
         n_axes=1, cu=None, cud=None, batch=0, used=None, tq=5, hq=4, hkv=2, d=64, qo=P, ko=P, out=F32):
    return lib.sa_norm_rope(q, k, src, hq * d, d, hkv * d, d, qw, kw, wt, eps, freq, rot, axes, 0, pos,
                            n_axes, tq, host(cu), cud, batch, used, tq, hq, hkv, d, qo, ko, out, hq * d,
                            d, hkv * d, d, None, None)


def test_norm_rope_checks(lib):
    assert rope(lib, hq=0, hkv=0) == 1 and rope(lib, hq=-1) == 1 and rope(lib, hkv=-2) == 1
    assert rope(lib, d=0) == 6 and rope(lib, rot=66) == 6 and rope(lib, rot=63) == 6
    assert rope(lib, rot=-2) == 6
    assert rope(lib, tq=-1) == 4 and rope(lib, n_axes=-1) == 4
    by = dict(pos=None, n_axes=0, batch=2, cu=CU, cud=P, used=P)
    assert rope(lib, **{**by, "cu": None}) == 3
    assert rope(lib, **{**by, "cu": np.array([0, 3, 2], np.int64)}) == 3
    assert rope(lib, **{**by, "batch": 0}) == 3
    assert rope(lib, **{**by, "tq": 4}) == 4
    for name in ("src", "wt", "out"):
        assert rope(lib, **{name: E4M3}) == 11
    assert rope(lib, eps=-1e-9) == 11 and rope(lib, eps=float("nan")) == 11
    assert rope(lib, **by, axes=P) == 11
    assert rope(lib, d=264) == 10
    for name in ("q", "k", "qo", "ko", "freq", "pos"):
        assert rope(lib, **{name: None}) == 11, name
    assert rope(lib, **{**by, "cud": None}) == 11 and rope(lib, **{**by, "used": None}) == 11
    assert rope(lib, tq=0, q=None, k=None) == 0
    # the order: what comes first is told first
    assert rope(lib, hq=0, hkv=0, d=0, tq=-1) == 1 and rope(lib, d=264, src=7) == 11


def load(lib, kp=P, vp=P, ks=P, vs=P, n=4, kind=INT8, bt=P, cols=2, cu=CU, cud=P, batch=2, tq=5,
         used=P, hkv=2, d=64, ps=16, k=P, v=P, out=F32, st=(128, 64, 128, 64)):
    return lib.sa_load_kv(kp, vp, ks, vs, n, kind, bt, cols, host(cu), cud, batch, tq, used, hkv, d, ps,
                          k, v, out, *st, None, None)


def test_load_checks(lib):
    assert load(lib, hkv=0) == 1
    assert load(lib, d=0) == 2 and load(lib, ps=0) == 2
    assert load(lib, cu=None) == 3 and load(lib, cu=np.array([1, 3, 5], np.int64)) == 3
    assert load(lib, tq=6) == 4 and load(lib, n=-1) == 4 and load(lib, cols=-1) == 4
    assert load(lib, out=INT8) == 11 and load(lib, kind=4) == 11 and load(lib, kind=-1) == 11
    assert load(lib, d=72) == 10 and load(lib, d=272) == 10 and load(lib, d=60, kind=BF16) == 10
    for name in ("kp", "vp", "ks", "vs", "bt", "cud", "used", "k", "v"):
        assert load(lib, **{name: None}) == 11, name
    for name in ("kp", "vp", "k", "v"):
        assert load(lib, **{name: P + 8}) == 11, name
    for i in range(4):
        st = [128, 64, 128, 64]
        st[i] += 2
        assert load(lib, st=st) == 11
        st[i] += 2
        assert load(lib, st=st, out=BF16) == 11
    assert load(lib, cu=np.array([0, 0, 0], np.int64), tq=0, k=None, v=None) == 0


def test_rows_of_an_output_that_share_elements(lib):
    for st in ((0, 64, 128, 64), (128, 0, 128, 64), (128, 64, 60, 64), (128, 64, 128, -32)):
        assert load(lib, st=st) == 11, st

    def rope_out(*st):
        return lib.sa_norm_rope(P, P, F32, 256, 64, 128, 64, P, P, F32, 1e-6, P, 64, None, 0, P, 1, 5, None,
                                None, 0, None, 5, 4, 2, 64, P, P, F32, *st, None, None)
    for st in ((0, 64, 128, 64), (256, 63, 128, 64), (256, 64, -1, 64), (256, 64, 128, 0)):
        assert rope_out(*st) == 11, st


def test_rows_of_an_output_that_meet_at_wide_strides(lib):
    """Token and head strides of a row or more each that still put one row's elements on another's, against
    all elements counted.  (Pages of 2^31 - 1 rows are refused after the strides: nothing is launched.)"""
    rng = np.random.default_rng(0)
    seen = [0, 0]
    for _ in range(2000):
        tokens, heads = int(rng.integers(1, 8)), int(rng.integers(8, 12))
        ts, hs = (int(x) * 64 * int(rng.choice([-1, 1])) for x in rng.integers(4, 60, 2))
        at = np.arange(tokens)[:, None] * ts + np.arange(heads) * hs
        meet = len(np.unique(at[..., None] + np.arange(256))) < at.size * 256
        for st in ((ts, hs, 1 << 20, 256), (1 << 20, 256, ts, hs)):
            got = load(lib, hkv=heads, d=256, ps=2 ** 31 - 1, cu=np.array([0, 0, tokens], np.int64), tq=tokens,
                       kind=F32, st=st)
            assert got == (11 if meet else 10), (tokens, heads, st)
        seen[meet] += 1
    assert min(seen) > 200
    # far strides: sums beyond 64 bits
    for st in ((2 ** 62, 2 ** 62, 4096, 256), (-(2 ** 63), 2 ** 62, 4096, 256)):
        assert load(lib, hkv=8, d=256, ps=2 ** 31 - 1, kind=F32, st=st) == 11
    assert load(lib, hkv=8, d=256, ps=2 ** 31 - 1, kind=F32, st=(2 ** 62, 256, 4096, 256)) == 10

    def rope_out(*st):
        return lib.sa_norm_rope(P, P, F32, 256, 64, 128, 64, P, P, F32, 1e-6, P, 64, None, 0, P, 1, 5, None,
                                None, 0, None, 5, 4, 2, 64, P, P, F32, *st, None, None)
    for st in ((64, 64, 128, 64), (128, 64, 128, 64), (256, 64, 100, 100), (90, 270, 128, 64)):
        assert rope_out(*st) == 11, st


def decode(lib, q=P, act=F32, kp=P, vp=P, ks=P, vs=P, n=4, kind=INT8, bt=P, cols=2, used=P, batch=2,
           hq=4, hkv=2, d=64, ps=16, window=0, out=P, lse=P, ws=P, nbytes=1 << 30):
    return lib.sa_decode_attention(q, act, kp, vp, ks, vs, n, kind, bt, cols, used, batch, hq, hkv, d, ps,
                                   0.1, window, out, lse, ws, nbytes, None, None)


def test_decode_checks(lib):
    assert decode(lib, hq=0) == 1 and decode(lib, hkv=0) == 1 and decode(lib, hq=5) == 1
    assert decode(lib, d=0) == 6
    assert decode(lib, batch=-1) == 4
    assert decode(lib, ps=0) == 2
    assert decode(lib, n=-1) == 4 and decode(lib, cols=-1) == 4 and decode(lib, window=-1) == 4
    assert decode(lib, act=INT8) == 11 and decode(lib, kind=4) == 11
    assert decode(lib, d=72) == 10 and decode(lib, d=272) == 10 and decode(lib, d=60, kind=F32) == 10
    assert decode(lib, batch=1 << 20, hq=1 << 12) == 10
    assert decode(lib, cols=1 << 20, ps=1024) == 10            # positions of a sequence: 2^29
    assert decode(lib, n=1 << 27, hkv=2, ps=16) == 10           # rows of the pool: below 2^32 - 1
    for name in ("q", "kp", "vp", "ks", "vs", "bt", "used", "out", "ws"):
        assert decode(lib, **{name: None}) == 11, name
    for name in ("q", "kp", "vp", "out", "ws"):
        assert decode(lib, **{name: P + 8}) == 11, name
    n = ctypes.c_size_t(0)
    assert lib.sa_decode_workspace_size(2, 4, 2, 64, ctypes.byref(n)) == 0 and n.value > 0
    assert decode(lib, nbytes=n.value - 1) == 11
    assert decode(lib, batch=0, q=None, out=None) == 0


def test_decode_workspace(lib):
    n = ctypes.c_size_t(0)
    assert lib.sa_decode_workspace_size(2, 5, 2, 64, ctypes.byref(n)) == 1
    assert lib.sa_decode_workspace_size(2, 4, 2, 0, ctypes.byref(n)) == 6
    assert lib.sa_decode_workspace_size(-1, 4, 2, 64, ctypes.byref(n)) == 4
    assert lib.sa_decode_workspace_size(2, 4, 2, 64, None) == 11
    # (what the kernels keep: never less with more heads or channels)
    last = 0
    for hq, d in ((8, 64), (16, 64), (16, 128), (32, 128), (32, 256)):
        assert lib.sa_decode_workspace_size(1, hq, 2, d, ctypes.byref(n)) == 0 and n.value >= last
        last = n.value
    # the same for every batch: it grows with the machine, not with the work
    sizes = set()
    for batch in (0, 1, 100, 10 ** 6):
        assert lib.sa_decode_workspace_size(batch, 64, 8, 128, ctypes.byref(n)) == 0
        sizes.add(n.value)
    assert len(sizes) == 1
