"""sa_load_kv against the definition: values are exact but for one rounding."""
import numpy as np
import pytest
import torch

import block_sparse_paged_csr_gb300 as sa
from _serving import TORCH, Cache, f64, on_gpu

pytestmark = pytest.mark.gpu


def check(qo, lens, kind, out, hkv=2, d=128, ps=16, seed=0, **kw):
    c = Cache(lens, kind, hkv, d, ps, seed=seed, **kw)
    cu = np.concatenate([[0], np.cumsum(qo)]).astype(np.int64)
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    got = sa.sa_load_kv(*c.pages, c.table, cu, on_gpu(cu, np.int64), c.used, dtype=TORCH[out],
                        status=status, **c.kw())
    assert int(status) == 0
    for which, g in enumerate(got):
        assert g.dtype == TORCH[out]
        for b, (n, m) in enumerate(zip(qo, lens)):
            first = max(m, 0) - n if max(m, 0) >= n else 0
            ref, _ = c.rows(b, list(range(first, first + n)), which)
            # code * scale is f32 arithmetic: the product's one rounding to f32 (exact under powers
            # of two), then one to the output's type
            ref = torch.from_numpy(ref.astype(np.float32)).to(TORCH[out])
            np.testing.assert_array_equal(f64(g[cu[b]:cu[b + 1]]), f64(ref))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3", "int8"])
def test_ragged(kind, out):
    """Single rows, whole sequences, none, page ends inside and at the ends, more rows than
    the sequence has (zeros)."""
    check([1, 5, 0, 33, 16, 1, 64, 9], [16, 21, 7, 33, 48, 100, 70, 4], kind, out, 3, 64)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3", "int8"])
@pytest.mark.parametrize("d,ps", [(16, 1), (48, 12), (128, 64), (256, 16), (80, 8), (208, 7), (96, 300)])
def test_sizes(kind, out, d, ps):
    check([40, 3], [45, 700], kind, out, 2, d, ps, seed=1)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_scales_of_any_kind(kind):
    check([30], [50], kind, "f32", seed=2, free_scales=True)
    check([30], [50], kind, "bf16", seed=2, free_scales=True)


def test_head_dim_of_8():
    check([20], [33], "bf16", "f32", 1, 8)
    check([20], [33], "f32", "bf16", 5, 24)


def test_absent_pages_and_short_tables():
    check([60, 5], [60, 5], "bf16", "f32", drop=[(0, 1), (0, 3)])
    check([60, 5], [60, 5], "int8", "bf16", drop=[(0, 0), (1, 0)])
    # a length past the table's columns
    c = Cache([20], "bf16", 2, 64, 16)
    cu = np.array([0, 40])
    k, v = sa.sa_load_kv(*c.pages, c.table, cu, on_gpu(cu, np.int64), on_gpu([50], np.int32))
    # (its two pages hold 32 rows, those behind the 20th NaN: the length says that they are rows)
    c.lens, c.values = [32], [f64(p) for p in c.pages]
    ref, _ = c.rows(0, list(range(10, 50)), 0)
    np.testing.assert_array_equal(f64(k), ref)


def test_a_page_outside_the_pool_is_reported():
    c = Cache([40], "f32", 1, 32, 16)
    c.table[0, 1] = c.pages[0].shape[0]
    c.bt[0, 1] = -1        # (what is expected: as if absent)
    cu = np.array([0, 40])
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    k, v = sa.sa_load_kv(*c.pages, c.table, cu, on_gpu(cu, np.int64), c.used, status=status)
    assert int(status) == 4
    for which, g in enumerate((k, v)):
        np.testing.assert_array_equal(f64(g), c.rows(0, list(range(40)), which)[0])


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3", "int8"])
def test_what_the_store_wrote(kind):
    """The store's rows come back: exactly from an f32 cache, else as the cache holds
    them; read into strided rows, with nothing else touched."""
    qo, lens, hkv, d, ps = [17, 1, 40], [30, 64, 40], 2, 64, 16
    cu = np.concatenate([[0], np.cumsum(qo)])
    c = Cache(lens, kind, hkv, d, ps, poison=False)
    x = torch.randn((int(cu[-1]), 2 * hkv, d), device="cuda")
    args = (c.table, cu, on_gpu(cu, np.int64), c.used)
    sa.sa_store_kv(x[:, :hkv], x[:, hkv:], *c.pages, *args, **c.kw())
    wide = torch.full((int(cu[-1]) + 1, 2 * hkv + 1, d), 9.0, device="cuda")
    k, v = sa.sa_load_kv(*c.pages, *args, k=wide[:-1, 1:hkv + 1], v=wide[:-1, hkv + 1:], **c.kw())
    assert (wide[:, 0] == 9.0).all() and (wide[-1] == 9.0).all()
    assert k.data_ptr() == wide[:, 1].data_ptr()
    for got, ref in ((k, x[:, :hkv]), (v, x[:, hkv:])):
        if kind == "f32":
            assert torch.equal(got, ref)
        elif kind == "bf16":
            assert torch.equal(got, ref.bfloat16().float())
        else:
            # half a step of a code, with the page's largest magnitude below 2 QMAX scales
            # (old rows of the page have the larger scale: their own, 2^-4 times at most 448 or 127)
            top = torch.maximum(ref.abs().amax(), torch.tensor(28.0 if kind == "e4m3" else 8.0))
            assert ((got - ref).abs() <= top * (2.0 ** -4 if kind == "e4m3" else 2.0 ** -7)).all()
    again = sa.sa_load_kv(*c.pages, *args, dtype=torch.bfloat16, **c.kw())
    assert torch.equal(again[0], k.bfloat16()) and torch.equal(again[1], v.bfloat16())


def test_graph():
    c = Cache([30, 50], "int8", 2, 64, 16)
    cu = np.array([0, 10, 60])
    cud = on_gpu(cu, np.int64)
    k, v = sa.sa_load_kv(*c.pages, c.table, cu, cud, c.used, **c.kw())
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sa.sa_load_kv(*c.pages, c.table, cu, cud, c.used, k=k2, v=v2, **c.kw())
    g.replay()
    assert torch.equal(k, k2) and torch.equal(v, v2)


def test_strides_of_a_single_row_say_nothing():
    """One row of one head out of a tensor of odd sizes."""
    c = Cache([30], "bf16", 1, 64, 16)
    cu = np.array([0, 1])
    wide = torch.zeros((3, 3, 65), device="cuda")
    k, v = (wide[i:i + 1].as_strided((1, 1, 64), (195, 65, 1), 256 * i) for i in (0, 1))
    sa.sa_load_kv(*c.pages, c.table, cu, on_gpu(cu, np.int64), c.used, k=k, v=v)
    for which, g in enumerate((k, v)):
        np.testing.assert_array_equal(f64(g), c.rows(0, [29], which)[0])
    rows = torch.zeros((1, 1, 64), device="cuda").expand(2, 1, 64)
    cu = np.array([0, 2])
    with pytest.raises(sa.SAError):
        sa.sa_load_kv(*c.pages, c.table, cu, on_gpu(cu, np.int64), c.used, k=rows, v=rows)


def test_refusals():
    c = Cache([30], "int8", 2, 64, 16)
    cu = np.array([0, 30])
    cud = on_gpu(cu, np.int64)

    def no(kind, pages=c.pages, cu=cu, cud=cud, **kw):
        with pytest.raises(kind):
            sa.sa_load_kv(*pages, c.table, cu, cud, c.used, **{**c.kw(), **kw})
    no(ValueError, k_scales=None)
    no(ValueError, v_scales=c.scales[0][:1])
    no(TypeError, dtype=torch.float16)
    no(TypeError, pages=[p.to(torch.int32) for p in c.pages])
    no(ValueError, pages=(c.pages[0], c.pages[1][:1]))
    no(ValueError, k=torch.empty((29, 2, 64), device="cuda"))
    no(ValueError, k=torch.empty((30, 2, 64), device="cuda"),
       v=torch.empty((30, 2, 64), device="cuda", dtype=torch.bfloat16))
    no(sa.SAError, k=torch.empty((30, 2, 65), device="cuda")[:, :, 1:])
    no(sa.SAError, cu=np.array([0, -1]))
    no(ValueError, cu=np.array([0, 3, 30]))
    odd = [torch.zeros((2, 1, 16, 24), dtype=torch.int8, device="cuda") for _ in range(2)]
    with pytest.raises(sa.SAError):
        sa.sa_load_kv(*odd, c.table, cu, cud, c.used, k_scales=torch.ones((2, 1), device="cuda"),
                      v_scales=torch.ones((2, 1), device="cuda"))
