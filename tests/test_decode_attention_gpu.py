"""sa_decode_attention against its formula in 64 bits."""
import math

import numpy as np
import pytest
import torch

import block_sparse_paged_csr_gb300 as sa
from _serving import HALF, TORCH, Cache, f64, on_gpu

pytestmark = pytest.mark.gpu
KINDS = ["f32", "bf16", "e4m3", "int8"]


def reference(c, q, scale, window):
    """Per (sequence, q-head): output, lse, sum p |v| / l per channel, the largest sum
    |q k| scale of a key (what the errors scale with), and what lies below the
    arithmetic's range (see check)."""
    batch, hq, d = q.shape
    g = hq // c.hkv
    out = np.zeros((batch, hq, d))
    size = np.zeros((batch, hq, d))
    lse = np.full((batch, hq), -np.inf)
    big, low = np.zeros((batch, hq)), np.zeros((batch, hq))
    for b in range(batch):
        n = c.lens[b]
        pos = list(range(max(0, n - window) if window else 0, min(n, c.bt.shape[1] * c.ps)))
        k, there = c.rows(b, pos, 0)
        v, _ = c.rows(b, pos, 1)
        vs = c.v_scales(b, pos)[there]
        k, v = k[there], v[there]
        if not len(k):
            continue
        for h in range(hq):
            s = k[:, h // g] @ q[b, h] * scale
            big[b, h] = (np.abs(k[:, h // g]) @ np.abs(q[b, h])).max() * abs(scale)
            m = s.max()
            p = np.exp(s - m)
            lse[b, h] = m + np.log(p.sum())
            p /= p.sum()
            out[b, h] = p @ v[:, h // g]
            size[b, h] = p @ np.abs(v[:, h // g])
            low[b, h] = len(k) * 2.0 ** -117 * np.abs(v[:, h // g]).max()
            if c.eight:
                top = (p * np.abs(vs[:, h // g])).max()
                low[b, h] += len(k) * 2.0 ** -28 * top * (128 if c.kind == "int8" else 448)
    return out, lse, size, big, low


def check(c, hq, act="f32", window=0, seed=0, qscale=1.0, scale=None, **kw):
    """A score's error: d + 16 roundings of sums of at most big (products of operands split
    into 22 bits or more count 4 of them), doubled for the tensor cores' cut additions; the score
    in base 2 has 24 bits, 3 2^-24 of its size.  That is an error of p; ex2 and the
    parts of p count 2^-21; sums over n keys in 8 or more chains n / 8 2^-24, and the merges
    64 2^-24.  l and o have it both.  bf16 queries: p in 11 bits or more, 2^-11, and the output's
    half step.  Below the range: a p under 2^-126 is 0, where the largest counts 2^-8 or more
    (the reference of the exponents may stand 2^7 and a step above it): 2^-117 a key.  Over 8 bits the
    product p vs goes to two f16 parts, whose last unit is 2^-24, half of it lost; the largest
    product counts more than 2^3 there: 2^-28 of it a key, times the largest code."""
    scale = 1.0 / math.sqrt(c.d) if scale is None else scale
    rng = np.random.default_rng(seed)
    q = torch.from_numpy(rng.standard_normal((len(c.lens), hq, c.d)) * qscale).cuda().to(TORCH[act])
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    out, lse = sa.sa_decode_attention(q, *c.pages, c.table, c.used, scale, window=window,
                                      status=status, **c.kw(), **kw)
    assert int(status) == 0 and out.dtype == q.dtype
    ref, rlse, size, big, low = reference(c, f64(q), scale, window)
    n = max(max(c.lens), 1)
    u = 2.0 ** -24
    ds = 2 * (c.d + 16) * u * big + 3 * u * (big + 1)
    part = 2 * ds + 2.0 ** -21 + (n / 4 + 128) * u
    tol = part[..., None] * size + HALF[out.dtype] * np.abs(ref) + (
        2.0 ** -11 * size if act == "bf16" else 0) + low[..., None]
    err = np.abs(f64(out) - ref)
    assert np.isfinite(f64(out)).all()
    assert (err <= tol).all(), f"{(err / np.maximum(tol, 1e-300)).max():.2f} of tol"
    got = f64(lse)
    np.testing.assert_array_equal(np.isfinite(got), np.isfinite(rlse))
    live = np.isfinite(rlse)
    assert (got[~live] == -np.inf).all()
    lerr = np.abs(got[live] - rlse[live])
    assert (lerr <= (part + 4 * u * np.abs(np.where(live, rlse, 0)))[live]).all(), lerr.max()
    return out, lse, q


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
def test_ragged(kind, act):
    """Lengths of nothing, one, page and tile ends, one below and above them."""
    lens = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 200, 0, 511, 1000]
    check(Cache(lens, kind, 2, 128, 16, extra_cols=1), 8, act)


@pytest.mark.parametrize("g", [1, 2, 3, 7, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("kind", KINDS)
def test_heads(kind, g):
    """All numbers of q-heads for a kv head, past a row tile of the MMA too."""
    for act in ("f32", "bf16"):
        check(Cache([70, 301], kind, 3, 64, 16, seed=g), 3 * g, act)


@pytest.mark.parametrize("d", [128, 200, 256])
@pytest.mark.parametrize("g", [9, 16, 20])
@pytest.mark.parametrize("kind", KINDS)
def test_many_heads_of_other_dims(kind, g, d):
    """Every instance with 16 query rows, whole pairs and cut ones."""
    d = d if kind in ("f32", "bf16") else d // 16 * 16
    for act in ("f32", "bf16"):
        check(Cache([41, 0, 700], kind, 2, d, 16, seed=g), 2 * g, act)


@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 240, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_head_dims(kind, d):
    check(Cache([130, 1, 77], kind, 2, d, 16, seed=d), 6)
    check(Cache([130, 1, 77], kind, 1, d, 16, seed=d), 12, "bf16")


@pytest.mark.parametrize("d", [8, 24, 40, 120, 200, 248])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_odd_head_dims(kind, d):
    check(Cache([130, 1, 77], kind, 2, d, 16, seed=d), 4)


@pytest.mark.parametrize("ps", [1, 3, 8, 12, 16, 64, 100, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_page_sizes(kind, ps):
    check(Cache([1, 99, 300, 257], kind, 2, 64, ps, seed=ps, free_scales=True), 4)


@pytest.mark.parametrize("window", [1, 5, 16, 33, 100, 5000])
@pytest.mark.parametrize("kind", KINDS)
def test_windows(kind, window):
    check(Cache([0, 1, 40, 99, 300, 257], kind, 2, 128, 16, seed=window), 6, window=window)


@pytest.mark.parametrize("kind", KINDS)
def test_absent_pages(kind):
    """Pages that the table does not have, whole sequences and windows of them."""
    c = Cache([100, 16, 64, 300], kind, 2, 128, 16, drop=[(0, 0), (0, 3), (1, 0), (2, 3), (3, 17), (3, 18)])
    check(c, 4)
    check(c, 4, window=16)


@pytest.mark.parametrize("kind", KINDS)
def test_one_long_sequence_is_split(kind):
    """Over all SMs and joined; scores of a large spread, so that the maxima of the parts
    differ."""
    check(Cache([30011], kind, 1, 64, 64, poison=False), 5, qscale=4.0)


@pytest.mark.parametrize("batch", [1, 150, 257, 1100])
def test_many_sequences(batch):
    lens = np.random.default_rng(batch).integers(0, 90, batch)
    check(Cache(lens, "e4m3", 2, 64, 16, poison=False), 4)
    check(Cache(lens, "f32", 1, 64, 16, poison=False), 2)


@pytest.mark.parametrize("kind", KINDS)
def test_large_and_small_scores(kind):
    c = Cache([333, 40], kind, 2, 128, 16)
    check(c, 4, qscale=100.0)
    check(c, 4, qscale=1e-4)
    check(c, 4, scale=0.0)
    check(c, 4, scale=-1.0)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_scales_far_apart(kind):
    """Pages of large and tiny scales: the values of a page that holds all of the softmax
    count, however small its V scale."""
    c = Cache([200, 96], kind, 1, 64, 16)
    n = c.scales[0].shape[0]
    rng = np.random.default_rng(3)
    for i, spread in ((0, 3), (1, 30)):
        s = on_gpu(2.0 ** rng.integers(-spread, spread, (n, 1)), np.float32)
        s = torch.where(torch.isnan(c.scales[i]), c.scales[i], s * (2.0 ** -8 if i == 0 else 1.0))
        codes = f64(c.pages[i])
        codes[~np.isfinite(codes)] = 0
        c.scales[i] = s
        c.values[i] = codes * np.nan_to_num(f64(s))[:, :, None, None]
    check(c, 4, qscale=3.0)


def test_the_scale_of_an_absent_page_is_not_read():
    c = Cache([64], "int8", 1, 64, 16, drop=[(0, 1)])
    c.scales = [torch.where(torch.arange(s.shape[0], device="cuda")[:, None] == 0, math.nan, s)
                for s in c.scales]
    check(c, 2)


def test_a_page_outside_the_pool_is_reported():
    c = Cache([64], "bf16", 1, 64, 16, drop=[(0, 1)])
    c.table[0, 1] = c.pages[0].shape[0]
    q = torch.randn((1, 2, 64), device="cuda")
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    out, _ = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1, status=status)
    assert int(status) == 4
    ref = reference(c, f64(q), 0.1, 0)[0]
    np.testing.assert_allclose(f64(out), ref, atol=1e-5)


def test_lengths_past_the_table():
    """At most the columns' positions; a window still ends at the length."""
    c = Cache([40], "f32", 1, 64, 8)
    q = torch.randn((1, 2, 64), device="cuda")
    used = on_gpu([1000], np.int32)
    out, lse = sa.sa_decode_attention(q, *c.pages, c.table, used, 0.1)
    same, _ = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1)
    assert torch.equal(out, same)
    out, lse = sa.sa_decode_attention(q, *c.pages, c.table, used, 0.1, window=100)
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = sa.sa_decode_attention(q, *c.pages, c.table, on_gpu([-7], np.int32), 0.1)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_windows_of_lengths_up_to_the_largest(kind, d):
    """A window behind the table's columns holds no keys, wherever it begins: its positions, rounded up
    to tiles, would pass 2^31.  One that reaches back into the table holds what is there."""
    top = 2 ** 31 - 1
    c = Cache([40, 40, 33, 40, 7], kind, 2, d, 16, seed=d)
    q = torch.randn((5, 4, d), device="cuda")
    for window in (1, 2, 7, 16, 30, 31, 32, 100):
        used = on_gpu([top, top - 1, 33, top - 15, 7], np.int32)
        status = torch.zeros(1, dtype=torch.int64, device="cuda")
        out, lse = sa.sa_decode_attention(q, *c.pages, c.table, used, 0.1, window=window, status=status,
                                          **c.kw())
        # (sequences without keys cut the work alike)
        same, slse = sa.sa_decode_attention(q, *c.pages, c.table, on_gpu([0, 0, 33, 0, 7], np.int32), 0.1,
                                            window=window, **c.kw())
        assert int(status) == 0 and torch.equal(out, same) and torch.equal(lse, slse)
        assert (out[[0, 1, 3]] == 0).all() and torch.isneginf(lse[[0, 1, 3]]).all()
    c = Cache([48, 40, 33, 48, 7], kind, 2, d, 16, seed=d, poison=False)
    for far, window, near, short in (([top, 40, 33, top, 7], top, c.lens, 0),
                                     ([1000, 18, 17, 1000, 7], 970, [48, 18, 17, 48, 7], 18)):
        out, lse = sa.sa_decode_attention(q, *c.pages, c.table, on_gpu(far, np.int32), 0.1, window=window,
                                          **c.kw())
        same, slse = sa.sa_decode_attention(q, *c.pages, c.table, on_gpu(near, np.int32), 0.1,
                                            window=short, **c.kw())
        assert torch.equal(out, same) and torch.equal(lse, slse)


@pytest.mark.parametrize("kind", KINDS)
def test_repeats_and_shared_workspace(kind):
    """The same bits again; one workspace for calls of other sizes, whatever it holds."""
    a = Cache([5000, 3, 900], kind, 2, 128, 16, poison=False)
    b = Cache([10, 70000], kind, 1, 64, 64, poison=False, seed=5)
    ws = sa.allocate_decode_workspace(3, 32, 2, 128, "cuda")
    ws.fill_(0xFF)
    qa, qb = torch.randn((3, 8, 128), device="cuda"), torch.randn((2, 5, 64), device="cuda")
    first = None
    for _ in range(3):
        x = sa.sa_decode_attention(qa, *a.pages, a.table, a.used, 0.1, workspace=ws, **a.kw())
        y = sa.sa_decode_attention(qb, *b.pages, b.table, b.used, 0.1, workspace=ws, **b.kw())
        got = [t.clone() for t in (*x, *y)]
        first = first or got
        assert all(torch.equal(s, t) for s, t in zip(first, got))


def test_graphs_replayed_over_other_lengths():
    """A captured call follows the lengths on the device, from nothing to all of the
    table; two graphs take turns with one workspace."""
    c = Cache([4000, 4000], "bf16", 2, 64, 16, poison=False)
    q = torch.randn((2, 4, 64), device="cuda")
    ws = sa.allocate_decode_workspace(2, 4, 2, 64, "cuda")
    outs, graphs = [], []
    for window in (0, 50):
        out, lse = torch.empty_like(q), torch.empty((2, 4), device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.125, window=window, out=out, lse=lse,
                                   workspace=ws)
        outs.append((out, lse))
        graphs.append(g)
    for lens in ([0, 4000], [17, 1], [3999, 0], [2500, 64]):
        c.used.copy_(on_gpu(lens, np.int32))
        for g in graphs:
            g.replay()
        for (out, lse), window in zip(outs, (0, 50)):
            x, y = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.125, window=window)
            assert torch.equal(out, x) and torch.equal(lse, y)


def test_streams_and_no_lse():
    c = Cache([700, 20], "int8", 2, 128, 16)
    q = torch.randn((2, 8, 128), device="cuda", dtype=torch.bfloat16)
    out, lse = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1, **c.kw())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x, none = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1, with_lse=False, stream=side,
                                     **c.kw())
    torch.cuda.current_stream().wait_stream(side)
    assert none is None and torch.equal(x, out)


def test_equals_sparse_attention_over_all_blocks():
    """The same numbers, up to rounding, as sa_attention with every block selected."""
    c = Cache([300, 64, 127], "e4m3", 2, 128, 16, poison=False)
    hq, bs = 8, 64
    cols = -(-c.bt.shape[1] // (bs // 16)) * (bs // 16)
    table = torch.full((3, cols), -1, dtype=torch.int32, device="cuda")
    table[:, :c.bt.shape[1]] = c.table
    sel = torch.arange(cols // 4, dtype=torch.int32, device="cuda").repeat(3, 2, 1)
    sel[sel * bs >= c.used[:, None, None]] = -1
    q = torch.randn((3, hq, 128), device="cuda")
    cu = np.arange(4)
    ref, rlse, _, _ = sa.sa_attention(q, *c.pages, sel.contiguous(), cu, on_gpu(cu, np.int64), c.used, table,
                                      hq, 2, 128, bs, 16, 0.1, True, **c.kw())
    out, lse = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1, **c.kw())
    torch.testing.assert_close(out, ref, rtol=1e-5, atol=1e-5)
    torch.testing.assert_close(lse, rlse, rtol=1e-5, atol=1e-5)


def test_no_pool_and_no_columns():
    """A cache without a page, a table without a column: nobody has keys."""
    q = torch.randn((2, 4, 64), device="cuda")
    none = torch.empty((0, 2, 16, 64), device="cuda")
    for table in (torch.zeros((2, 3), dtype=torch.int32, device="cuda"),
                  torch.zeros((2, 0), dtype=torch.int32, device="cuda")):
        out, lse = sa.sa_decode_attention(q, none, none, table, on_gpu([0, 40], np.int32), 0.1)
        assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_scales_of_zero_and_at_the_ends(kind):
    """Rows of zeros have scale 0: all keys count alike.  Values at both ends of f32."""
    c = Cache([90], kind, 1, 64, 16, poison=False)
    c.scales[0].zero_()
    q = torch.randn((1, 2, 64), device="cuda")
    out, lse = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1, **c.kw())
    v, _ = c.rows(0, list(range(90)), 1)
    # f32 sums of 90 products with p = 1, at most 90 half steps; codes of up to 448 scales
    np.testing.assert_allclose(f64(out)[0, 0], v.mean(0)[0], atol=90 * 2.0 ** -24 * 448 * 2.0 ** -4)
    assert abs(float(lse[0, 0]) - math.log(90)) < 1e-5
    for e in (-126, -60, 60, 116):
        c.scales[1].fill_(2.0 ** e)
        big, _ = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1, **c.kw())
        c.scales[1].fill_(1.0)
        one, _ = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1, **c.kw())
        # (a power of two: the same codes times it; at 2^-126 results leave f32's normal range)
        np.testing.assert_allclose(f64(big), f64(one) * 2.0 ** e, rtol=2.0 ** -20, atol=2.0 ** -148)
    c.scales[1].zero_()
    out, _ = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1, **c.kw())
    assert (out == 0).all()


def test_a_query_that_is_no_number_stays_its_own():
    """NaN in one row leaves the others, whole pairs and merged ones alike, and comes out."""
    for lens in ([5, 40], [5, 60000]):
        c = Cache(lens, "bf16", 1, 64, 16, poison=False)
        q = torch.randn((2, 4, 64), device="cuda")
        ref, rlse = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1)
        q[1, 2, 7] = math.nan
        out, lse = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1)
        assert torch.isnan(out[1, 2]).all() and torch.isnan(lse[1, 2])
        keep = torch.ones((2, 4), dtype=torch.bool, device="cuda")
        keep[1, 2] = False
        assert torch.equal(out[keep], ref[keep]) and torch.equal(lse[keep], rlse[keep])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_a_key_or_value_that_is_no_number_stays_its_own(kind):
    """NaN in one row of K comes out for its sequence and kv head, in one row of V for its channel,
    whole pairs and merged ones alike; all else keeps its bits."""
    for lens, b, at in (([5, 40, 33], 1, 17), ([5, 60000, 33], 1, 41234)):
        c = Cache(lens, kind, 2, 64, 16, poison=False)
        q = torch.randn((3, 8, 64), device="cuda")
        ref, rlse = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1)
        page = int(c.bt[b, at // 16])
        old = c.pages[1][page, 1, at % 16, 3].clone()
        c.pages[1][page, 1, at % 16, 3] = math.nan
        out, lse = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1)
        hit = torch.zeros((3, 8, 64), dtype=torch.bool, device="cuda")
        hit[b, 4:, 3] = True
        assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], ref[~hit])
        assert torch.equal(lse, rlse)
        c.pages[1][page, 1, at % 16, 3] = old
        c.pages[0][page, 1, at % 16, 3] = math.nan
        out, lse = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1)
        hit[b, 4:] = True
        assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], ref[~hit])
        rows = hit.any(2)
        assert torch.isnan(lse[rows]).all() and torch.equal(lse[~rows], rlse[~rows])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 15, 100])
def test_rows_before_a_window_are_not_read(kind, window):
    """No numbers in the rows before it, within the tile where it starts too, nor in the scales of
    pages that lie before it as a whole."""
    lens, ps = [90, 257, 300, 31], 16
    c = Cache(lens, kind, 2, 64, ps, seed=window)
    for b, n in enumerate(lens):
        for p in range(max(n - window, 0)):
            page = int(c.bt[b, p // ps])
            for x in c.pages:
                if kind == "int8":
                    x[page, :, p % ps] = -128
                elif kind == "e4m3":
                    x.view(torch.uint8)[page, :, p % ps] = 0x7F
                else:
                    x[page, :, p % ps] = math.nan
            if c.eight and p % ps == ps - 1:
                for s in c.scales:
                    s[page] = math.nan
    for act in ("f32", "bf16"):
        check(c, 6, act, window=window)


@pytest.mark.parametrize("kind", KINDS)
def test_softmax_scales_of_any_sign(kind):
    c = Cache([0, 40, 300], kind, 2, 64, 16)
    for scale in (0.0, -0.125, 2.0 ** -60, 1.5):
        check(c, 6, scale=scale)


def test_refusals():
    c = Cache([30, 7], "int8", 2, 64, 16)
    q = torch.randn((2, 4, 64), device="cuda")

    def no(kind, q=q, pages=c.pages, table=c.table, used=c.used, **kw):
        with pytest.raises(kind):
            sa.sa_decode_attention(q, *pages, table, used, 0.1, **{**c.kw(), **kw})
    no(TypeError, q=q.half())
    no(TypeError, q=None)
    no(ValueError, q=q.cpu())
    no(ValueError, q=q[:, :, :32])
    no(ValueError, q=q[0])
    no(sa.SAError, q=q[:, :3].contiguous())
    no(ValueError, q=q.transpose(0, 1))
    no(TypeError, table=c.table.long())
    no(ValueError, table=c.table[:1])
    no(ValueError, used=c.used[:1])
    no(TypeError, used=c.used.long())
    no(ValueError, k_scales=None)
    no(ValueError, v_scales=c.scales[1].T)
    no(sa.SAError, window=-1)
    no(ValueError, out=torch.empty((2, 3, 64), device="cuda"))
    no(TypeError, out=torch.empty((2, 4, 64), device="cuda", dtype=torch.bfloat16))
    no(ValueError, lse=torch.empty(7, device="cuda"))
    no(sa.SAError, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    no(TypeError, workspace=torch.empty(800, device="cuda"))
    no(ValueError, out=q)
    out, lse = sa.sa_decode_attention(q[:0], *c.pages, c.table[:0], c.used[:0], 0.1, **c.kw())
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("kind", KINDS)
def test_long_sums_do_not_drift(kind):
    """Sums over many tiles by one warp: 256 sequences of 65536 keys that share their pages, all
    values near 1, so that a sum which is cut at every step (2^-25 of it on average) shows as an output
    below the true one.  A warp adds 256 * 2 * 65536 / (1824 * 32) = 575 tiles or more of 32 keys:
    cut, they would leave 575 2^-26 = 9e-6 missing (16 keys a tile: 1.7e-5).  What may be
    missing: a tile's own products are cut at most 3 times, 3 2^-24 = 2e-7; rounding
    errors of the additions have no sign, at most half a step each, and their mean over 4096 x 64
    outputs vanishes beside it.  ex2 is off by 2^-22 in numerator and denominator alike.  1e-6."""
    batch, hkv, g, n, d, ps = 256, 2, 2, 65536, 64, 64
    gen = torch.Generator(device="cuda").manual_seed(4)
    shape = (n // ps, hkv, ps, d)
    k = torch.randn(shape, generator=gen, device="cuda")
    v = 1 + 0.05 * torch.randn(shape, generator=gen, device="cuda")
    kw = {}
    if kind in ("e4m3", "int8"):
        k, v = (k * 30).to(TORCH[kind]), (v * 64).to(TORCH[kind])
        s = torch.full((n // ps, hkv), 2.0 ** -6, device="cuda")
        kw = dict(k_scales=s, v_scales=s)
    else:
        k, v = k.to(TORCH[kind]), v.to(TORCH[kind])
    kx, vx = (x.float().double() * (2.0 ** -6 if kw else 1) for x in (k, v))
    table = torch.arange(n // ps, dtype=torch.int32, device="cuda").repeat(batch, 1)
    q = torch.randn((batch, hkv * g, d), generator=gen, device="cuda")
    out, lse = sa.sa_decode_attention(q, k, v, table, torch.full((batch,), n, dtype=torch.int32, device="cuda"),
                                      0.125, **kw)
    for h in range(hkv):
        keys, vals = (x[:, h].reshape(n, d) for x in (kx, vx))
        x = q[:, h * g:(h + 1) * g].double().reshape(-1, d) @ keys.T * 0.125
        ref = torch.softmax(x, 1) @ vals
        got = out[:, h * g:(h + 1) * g].double().reshape(-1, d)
        assert abs(float(((got - ref) / ref).mean())) <= 1e-6
        # (rounding: 575 additions of half a step, 2^-25, at random: 24 2^-25, six of them)
        assert float(((got - ref).norm() / ref.norm())) <= 6 * 24 * 2.0 ** -25


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("f32", 64), ("int8", 256)])
def test_pages_far_into_a_pool(kind, d):
    """Pages whose bytes, and whose elements, lie beyond 2^32 from the pool's start."""
    hkv, ps = 8, 64
    per = hkv * ps * d
    n = 2 ** 32 // per + 300
    pools = [torch.zeros((n, hkv, ps, d), dtype=TORCH[kind], device="cuda") for _ in range(2)]
    kw = {}
    if kind == "int8":
        scales = torch.full((n, hkv), 2.0 ** -5, device="cuda")
        kw = dict(k_scales=scales, v_scales=scales)
    ids = torch.tensor([n - 1, n - 200, 3, n - 77], device="cuda")
    for p in pools:
        x = torch.randn((4, hkv, ps, d), device="cuda")
        p[ids] = ((x * 40).round().clamp(-127, 127) if kind == "int8" else x).to(TORCH[kind])
    table = ids.to(torch.int32).view(2, 2).contiguous()
    used = on_gpu([100, 128], np.int32)
    q = torch.randn((2, 16, d), device="cuda")
    out, lse = sa.sa_decode_attention(q, *pools, table, used, d ** -0.5, **kw)
    small = [p[ids] for p in pools]
    if kw:
        kw = dict(k_scales=scales[ids], v_scales=scales[ids])
    near = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    same, slse = sa.sa_decode_attention(q, *small, near, used, d ** -0.5, **kw)
    assert torch.equal(out, same) and torch.equal(lse, slse) and float(out.abs().max()) > 0
    cu = np.array([0, 100, 228])
    if kw:
        kw = dict(k_scales=scales, v_scales=scales)
    k, v = sa.sa_load_kv(*pools, table, cu, on_gpu(cu, np.int64), used, dtype=torch.float32, **kw)
    for got, p in ((k, small[0]), (v, small[1])):
        rows = torch.cat([p[:2].transpose(1, 2).reshape(-1, hkv, d)[:100], p[2:].transpose(1, 2).reshape(-1, hkv, d)])
        assert torch.equal(got, rows.float() * (2.0 ** -5 if kw else 1))


@pytest.mark.parametrize("g", [5, 12])
@pytest.mark.parametrize("kind", KINDS)
def test_one_long_sequence_of_bf16_queries_is_split(kind, g):
    """As above for bf16 queries, with 8 and 16 rows a tile: parts of differing references joined."""
    check(Cache([30011], kind, 1, 64, 64, poison=False, free_scales=True), g, "bf16", qscale=4.0)


def test_calls_side_by_side_from_two_threads():
    """Two host threads, a stream and a workspace each, calls of all three operators that overlap on the
    GPU: the bits of calls made alone."""
    import threading

    def work(i):
        kind, act = (("int8", torch.bfloat16), ("bf16", torch.float32))[i]
        c = Cache([3000, 5, 900], kind, 2, 128, 16, poison=False, seed=i)
        gen = torch.Generator(device="cuda").manual_seed(i)
        x = torch.randn((3, 10, 128), generator=gen, device="cuda").to(act)
        f = on_gpu(10000.0 ** (-np.arange(64) / 64), np.float32)
        cu = np.arange(4)
        cud, status = on_gpu(cu, np.int64), torch.zeros(1, dtype=torch.int64, device="cuda")
        stream, ws = torch.cuda.Stream(), sa.allocate_decode_workspace(3, 8, 2, 128, "cuda")

        def step(stream=None):
            q, _ = sa.sa_norm_rope(x[:, :8], x[:, 8:], None, None, f, cu_seqlens_q_host=cu, cu_seqlens_q=cud,
                                   used_kv_lens=c.used, status=status, stream=stream)
            out, lse = sa.sa_decode_attention(q, *c.pages, c.table, c.used, 0.1, workspace=ws, status=status,
                                              stream=stream, **c.kw())
            k, v = sa.sa_load_kv(*c.pages, c.table, cu, cud, c.used, status=status, stream=stream, **c.kw())
            return q, out, lse, k, v
        return step, stream, status

    both = [work(i) for i in range(2)]
    alone = [[t.clone() for t in step()] for step, _, _ in both]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def loop(i):
        try:
            step, stream, _ = both[i]
            for _ in range(40):
                got[i].append(step(stream))
        except Exception as e:          # (told by the main thread)
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for i in range(2):
        assert len(got[i]) == 40 and int(both[i][2]) == 0
        for one in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(one, alone[i]))
