"""sa_norm_rope against its formula in 64 bits."""
import numpy as np
import pytest
import torch

import block_sparse_paged_csr_gb300 as sa
from _serving import HALF, TORCH, f64, on_gpu

pytestmark = pytest.mark.gpu


def reference(x, w, freq, pos, eps, interleaved):
    """(result, size) of rows x [t, h, d] in 64 bits; pos [t, pairs].  size: |a| + |b| of
    a channel's pair, what its rounding errors scale with."""
    y = x if w is None else x / np.sqrt((x * x).mean(2, keepdims=True) + eps) * w
    size = np.abs(y)
    n = 0 if freq is None else len(freq)
    if n:
        t = (pos.astype(np.float64) * freq)[:, None]
        a, b = (np.arange(n) * 2, np.arange(n) * 2 + 1) if interleaved else (
            np.arange(n), np.arange(n) + n)
        ya, yb = y[..., a], y[..., b]
        y, size = y.copy(), size.copy()
        y[..., a] = ya * np.cos(t) - yb * np.sin(t)
        y[..., b] = ya * np.sin(t) + yb * np.cos(t)
        size[..., a] = size[..., b] = np.abs(ya) + np.abs(yb)
    return y, size


def close(got, ref, size):
    """Half a step of the output type, and f32 arithmetic: at most 24 additions in a
    lane's and the warp's sum of squares (half of their error reaches the root), rsqrt 2
    ulp, mean, weight and product 4, the angle's f32 rounding (pi 2^-25) and sincospi 4,
    rotation 3 roundings: 27 2^-24 in all; 40 leaves the second-order terms."""
    tol = HALF[got.dtype] * np.abs(ref) + 40 * 2.0 ** -24 * size
    err = np.abs(f64(got) - ref)
    assert np.isfinite(err).all() and (err <= tol).all(), f"{(err / np.maximum(tol, 1e-30)).max():.2f} of tol"


def freqs(rot, base=10000.0):
    return (base ** (-np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32)


def run(tq, hq, hkv, d, rot, src, out, interleaved=False, norm=True, axes=0, seed=0, base_pos=0,
        wt=None, inplace=False, pad=3, offset=0):
    rng = np.random.default_rng(seed)
    wide = hq + hkv + pad
    buf = torch.from_numpy(rng.standard_normal((tq, wide * d + offset)) * 2.0).cuda().to(TORCH[src])
    qkv = buf[:, offset:].unflatten(1, (wide, d))
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    w = None
    if norm:
        w = [torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).cuda().to(TORCH[wt or src])
             for _ in range(2)]
    f = freqs(rot)
    kw = dict(interleaved=interleaved, eps=1e-5)
    n = rot // 2
    if axes:
        pos = rng.integers(-50, 200000, (axes, tq))
        of = rng.integers(0, axes, n)
        kw.update(positions=on_gpu(pos, np.int32), freq_axes=on_gpu(of, np.int32))
        p = pos[of].T
    else:
        p1 = base_pos + rng.permutation(tq)
        kw.update(positions=on_gpu(p1, np.int32))
        p = np.repeat(p1[:, None], n, 1)
    before = f64(qkv).copy()
    if inplace:
        kw.update(q_out=q, k_out=k)
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    go, ko = sa.sa_norm_rope(q, k, None if w is None else w[0], None if w is None else w[1],
                             on_gpu(f, np.float32) if rot else None, out_dtype=TORCH[out],
                             status=status, **kw)
    assert int(status) == 0
    for got, x, i in ((go, before[:, :hq], 0), (ko, before[:, hq:hq + hkv], 1)):
        ref, size = reference(x, None if w is None else f64(w[i]), f.astype(np.float64), p, 1e-5,
                              interleaved)
        close(got, ref, size)
    if inplace:
        assert go.data_ptr() == q.data_ptr()
        np.testing.assert_array_equal(f64(qkv)[:, hq + hkv:], before[:, hq + hkv:])
    else:
        np.testing.assert_array_equal(f64(qkv), before)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("src,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
def test_types(src, out, interleaved):
    run(19, 6, 2, 128, 128, src, out, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 64), (256, 256), (96, 96), (80, 32),
                                   (80, 80), (72, 48), (24, 16), (16, 16), (8, 0), (256, 0),
                                   (128, 10), (36, 36), (6, 2), (1, 0), (250, 100), (200, 192)])
def test_head_sizes(d, rot, interleaved):
    """Both kernels: pieces of 8 channels, and any size."""
    run(11, 5, 3, d, rot, "bf16", "f32", interleaved, seed=1)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(16, 16), (64, 32), (80, 48), (256, 256), (256, 16), (144, 0),
                                   (48, 24), (24, 24), (200, 192)])
def test_head_sizes_of_bf16(d, rot, interleaved):
    """Pieces of 8 channels and of 4, the latter also where only the start or a stride forbids 8; more
    than one turn of a group over its heads."""
    run(11, 5, 3, d, rot, "bf16", "bf16", interleaved, seed=4)
    run(11, 5, 3, d, rot, "bf16", "bf16", interleaved, offset=4, seed=5)
    run(9, 5, 3, d, rot, "bf16", "bf16", interleaved, norm=False, seed=6)
    run(501, 70, 3, d, rot, "bf16", "bf16", interleaved, seed=7)


@pytest.mark.parametrize("tq,hq,hkv", [(1, 1, 1), (1, 64, 8), (3, 1, 0), (5, 0, 2), (700, 7, 1),
                                       (1025, 40, 8), (4, 300, 5)])
def test_counts(tq, hq, hkv):
    """One row, one kind of heads, few and many rows of a token (both ways to cut
    the work)."""
    if hq and hkv:
        run(tq, hq, hkv, 128, 128, "bf16", "bf16", seed=2)
        return
    x = torch.randn((tq, hq + hkv, 128), device="cuda")
    f = freqs(128)
    q, k = (x, None) if hq else (None, x)
    pos = np.arange(tq) * 1000
    got = sa.sa_norm_rope(q, k, None, None, on_gpu(f, np.float32), positions=on_gpu(pos, np.int32))
    ref, size = reference(f64(x), None, f.astype(np.float64), np.repeat(pos[:, None], 64, 1), 0, False)
    close(got[0] if hq else got[1], ref, size)
    assert got[1 if hq else 0] is None


@pytest.mark.parametrize("d,rot", [(128, 128), (128, 30)])
def test_axes(d, rot):
    for axes in (1, 3, 5):
        run(33, 4, 2, d, rot, "f32", "f32", axes % 2 == 1, axes=axes, seed=axes)


@pytest.mark.parametrize("base", [0, 131072, 2 ** 24 - 3, 2 ** 31 - 40, -(2 ** 31)])
def test_far_positions(base):
    run(31, 2, 1, 64, 64, "f32", "f32", base_pos=base, seed=3)


def test_without_norm_and_weights_of_another_type():
    run(9, 3, 3, 128, 64, "bf16", "bf16", norm=False)
    run(9, 3, 3, 128, 64, "bf16", "bf16", wt="f32")
    run(9, 3, 3, 40, 22, "f32", "f32", wt="bf16")


def test_frequencies_of_any_size():
    """From subnormal to several turns a step, and negative ones."""
    f = np.array([1e-42, 1e-30, 1e-3, 0.5, 1.0, 3.0, 6.5, 100.0, -0.25, 0.0, 2.0 ** -20, 1e5,
                  2.0 ** 40, 7.7, -1e-9, 0.1], np.float32)
    pos = np.array([0, 1, -1, 17, 1000, 131071, 2 ** 31 - 1, -2 ** 31])
    x = torch.randn((len(pos), 2, 32), device="cuda")
    got, _ = sa.sa_norm_rope(x, None, None, None, on_gpu(f, np.float32), positions=on_gpu(pos, np.int32))
    # a product of 32 and 24 bits in 64-bit turns: 2^-64 |p| of error, 2^-31 turns kept; the angle in
    # extended precision, its whole turns dropped (numpy's 64 bits alone lose them here)
    p = np.repeat(pos[:, None], 16, 1)
    turns = p.astype(np.longdouble) * f.astype(np.longdouble) / (2 * np.pi)
    if np.finfo(np.longdouble).nmant >= 63:
        two_pi = np.longdouble("6.2831853071795864769252867665590057684")
        turns = p.astype(np.longdouble) * f.astype(np.longdouble) / two_pi
    t = (2 * np.pi * (turns - np.rint(turns)).astype(np.float64))[:, None]
    xx = f64(x)
    a, b = xx[..., :16], xx[..., 16:]
    ref = np.concatenate([a * np.cos(t) - b * np.sin(t), a * np.sin(t) + b * np.cos(t)], 2)
    size = np.tile(np.abs(a) + np.abs(b), 2)
    ok = np.abs(p * f.astype(np.float64)) < 2.0 ** 26 if np.finfo(np.longdouble).nmant < 63 else (
        np.abs(p * f.astype(np.float64)) < 2.0 ** 34)
    # (the reference's own error: |turns| 2^-52, or 2^-63)
    ok = np.tile(ok, 2)[:, None] & np.ones_like(size, bool)
    err = np.abs(f64(got) - ref)
    assert np.isfinite(err).all()
    assert (err[ok] <= 40 * 2.0 ** -24 * size[ok]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_near_quarter_turns(interleaved):
    """The angle's own error, seen where cosine or sine is small: rows (1, 0) come out as both.  The angle
    is rounded to f32 within an eighth of a turn of the nearest quarter, 2^-28 turns, after products that
    are 2^-32 off (frequencies up to 256); sincospi's results are 2 ulp off, 2 2^-23 relative.  (Rounded
    as a part of a whole turn it would be 2^-26 off, and from frequencies of 4 on, without the product's
    lower bits, more.)  Positions whose turns lie near a quarter are looked for."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194989")
    f = np.array([1.0, 0.7, 0.01, 1e-4, -0.3, 5.0, 100.0, 250.0], np.float32)
    rng = np.random.default_rng(1)
    pos, turns = [], []
    for fi in f:
        x = np.concatenate([rng.integers(0, 2 ** 31, 20000), rng.integers(0, 4000, 500),
                            [0, 1, 2 ** 31 - 1, -2 ** 31]])
        t = x.astype(np.longdouble) * np.longdouble(fi) * 4 / (2 * np.pi)
        x = x[np.argsort(np.abs(t - np.rint(t)))[:60]]
        pos.append(x)
        turns.append([float((Decimal(int(p)) * Decimal(float(fi)) / two_pi) % 1) for p in x])
    pos = np.concatenate(pos)                       # [8 * 60] tokens, each for one of the pairs
    own = np.repeat(np.arange(8), 60)
    x = torch.zeros((len(pos), 1, 16), device="cuda")
    a, b = (slice(0, 16, 2), slice(1, 16, 2)) if interleaved else (slice(0, 8), slice(8, 16))
    x[..., a] = 1
    got, _ = sa.sa_norm_rope(x, None, None, None, on_gpu(f, np.float32), positions=on_gpu(pos, np.int32),
                             interleaved=interleaved)
    i = np.arange(len(pos))
    cos, sin = f64(got)[i, 0, a][i, own], f64(got)[i, 0, b][i, own]
    t = 2 * np.pi * np.concatenate(turns)
    angle = 2 * np.pi * (2.0 ** -28 + 2.0 ** -32)
    for y, ref, slope in ((cos, np.cos(t), np.sin(t)), (sin, np.sin(t), np.cos(t))):
        err, tol = np.abs(y - ref), angle * np.abs(slope) + 2.0 ** -22 * np.abs(ref) + 2.0 ** -50
        assert (err <= tol).all(), (err / tol).max()


def test_in_place_and_other_strides():
    run(21, 4, 2, 128, 128, "bf16", "bf16", inplace=True)
    run(21, 4, 2, 36, 20, "f32", "f32", True, inplace=True)
    # rows that do not start on 16 bytes
    run(21, 4, 2, 128, 128, "bf16", "bf16", offset=1)
    # heads outside tokens in the output
    x = torch.randn((13, 4, 64), device="cuda", dtype=torch.bfloat16)
    out = torch.full((4, 13, 64), 7.0, device="cuda")
    pos = torch.arange(13, dtype=torch.int32, device="cuda")
    f = on_gpu(freqs(64), np.float32)
    sa.sa_norm_rope(x, None, None, None, f, positions=pos, q_out=out.transpose(0, 1))
    same, _ = sa.sa_norm_rope(x, None, None, None, f, positions=pos, out_dtype=torch.float32)
    assert torch.equal(out.transpose(0, 1), same)


@pytest.mark.parametrize("tq,hq,hkv", [(1, 40, 8), (300, 1, 1), (1, 1, 1)])
@pytest.mark.parametrize("src,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_strides_that_nothing_is_multiplied_by(src, out, tq, hq, hkv):
    """Of a single token or a single head: whatever they are, the same bits by the same kernel."""
    d = 128
    gen = torch.Generator(device="cuda").manual_seed(tq + hq)
    q, k = (torch.randn((tq, h, d), generator=gen, device="cuda").to(TORCH[src]) for h in (hq, hkv))
    w = torch.rand(d, generator=gen, device="cuda").to(TORCH[src])
    f = on_gpu(freqs(d), np.float32)
    pos = torch.arange(tq, dtype=torch.int32, device="cuda") + 100

    def odd(x):
        return x.as_strided(x.shape, (777 if tq == 1 else x.stride(0), 3 if x.shape[1] == 1 else d, 1))
    a, b = sa.sa_norm_rope(q, k, w, w, f, positions=pos, out_dtype=TORCH[out])
    qo, ko = (torch.empty(x.shape, dtype=TORCH[out], device="cuda") for x in (q, k))
    c, e = sa.sa_norm_rope(odd(q), odd(k), w, w, f, positions=pos, q_out=odd(qo), k_out=odd(ko))
    assert torch.equal(a, c) and torch.equal(b, e)


def test_positions_from_lengths():
    """The new tokens end at the sequence's length; sequences without new tokens, one
    shorter than its new tokens; both kernels; rows behind the last one stay."""
    qo, lens = [1, 0, 5, 70, 3], [9, 4, 5, 1000, 2]
    cu = np.concatenate([[0], np.cumsum(qo)]).astype(np.int64)
    tq = int(cu[-1])
    pos = np.concatenate([np.arange(n) + max(m - n, 0) for n, m in zip(qo, lens)])
    for d, rot in ((128, 128), (128, 12)):
        x = torch.randn((tq, 3, d), device="cuda")
        f = on_gpu(freqs(rot), np.float32)
        room = torch.full((tq + 2, 3, d), 5.0, device="cuda")
        got, _ = sa.sa_norm_rope(x, None, None, None, f, cu_seqlens_q_host=cu,
                                 cu_seqlens_q=on_gpu(cu, np.int64), used_kv_lens=on_gpu(lens, np.int32),
                                 q_out=room[:tq])
        same, _ = sa.sa_norm_rope(x, None, None, None, f, positions=on_gpu(pos, np.int32))
        assert torch.equal(got, same)
        assert (room[tq:] == 5.0).all()


def test_many_sequences_of_one_token():
    n = 2100
    lens = np.random.default_rng(0).integers(1, 100000, n)
    cu = np.arange(n + 1)
    x = torch.randn((n, 1, 64), device="cuda")
    f = on_gpu(freqs(64), np.float32)
    got, _ = sa.sa_norm_rope(x, None, None, None, f, cu_seqlens_q_host=cu,
                             cu_seqlens_q=on_gpu(cu, np.int64), used_kv_lens=on_gpu(lens, np.int32))
    same, _ = sa.sa_norm_rope(x, None, None, None, f, positions=on_gpu(lens - 1, np.int32))
    assert torch.equal(got, same)


@pytest.mark.parametrize("rot", [128, 20])
def test_tokens_far_into_a_tensor(rot):
    """Elements beyond 2^31 from the tensor's start, by both kernels."""
    tq, hq, d = 140001, 128, 128
    q = torch.empty((tq, hq, d), dtype=torch.bfloat16, device="cuda")
    q[-5:].normal_()
    q[:-5].zero_()
    f = on_gpu(freqs(rot), np.float32)
    pos = torch.arange(tq, dtype=torch.int32, device="cuda")
    w = torch.ones(d, device="cuda")
    got, _ = sa.sa_norm_rope(q, None, w, None, f, positions=pos)
    same, _ = sa.sa_norm_rope(q[-5:].contiguous(), None, w, None, f, positions=pos[-5:].contiguous())
    assert torch.equal(got[-5:], same) and float(same.abs().max()) > 0
    assert not got[:1000].any()


def test_an_axis_outside_is_reported():
    x = torch.randn((3, 1, 32), device="cuda")
    f = on_gpu(freqs(32), np.float32)
    pos = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    bad = torch.zeros(16, dtype=torch.int32, device="cuda")
    bad[3], bad[9] = 2, -1
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    got, _ = sa.sa_norm_rope(x, None, None, None, f, positions=pos, freq_axes=bad, status=status)
    assert int(status) == 4
    same, _ = sa.sa_norm_rope(x, None, None, None, f, positions=pos[0].contiguous())
    assert torch.equal(got, same)


def test_graph_and_streams():
    """Captured, and replayed over other contents; on a stream that is named."""
    x = torch.randn((8, 6, 128), device="cuda")
    f = on_gpu(freqs(128), np.float32)
    w = torch.rand(128, device="cuda")
    cu = np.arange(9)
    cud, used = on_gpu(cu, np.int64), on_gpu(np.arange(8) + 5, np.int32)
    kw = dict(cu_seqlens_q_host=cu, cu_seqlens_q=cud, used_kv_lens=used)
    q_out, k_out = torch.empty((8, 4, 128), device="cuda"), torch.empty((8, 2, 128), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sa.sa_norm_rope(x[:, :4], x[:, 4:], w, w, f, q_out=q_out, k_out=k_out, **kw)
    x.normal_()
    used += 100
    g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = sa.sa_norm_rope(x[:, :4], x[:, 4:], w, w, f, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, q_out) and torch.equal(b, k_out)


def test_refusals():
    x = torch.randn((4, 2, 32), device="cuda")
    f = on_gpu(freqs(32), np.float32)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")

    def no(kind, q=x, k=None, wq=None, fr=f, **kw):
        with pytest.raises(kind):
            sa.sa_norm_rope(q, k, wq, None, fr, **{"positions": pos, **kw})
    no(TypeError, q=x.half())
    no(TypeError, q=None)
    no(ValueError, q=x.cpu())
    no(ValueError, q=x.transpose(1, 2))
    no(ValueError, k=x[:3])
    no(ValueError, k=x.bfloat16())
    no(ValueError, q=x[:, 0])
    no(TypeError, fr=f.double())
    no(TypeError, wq=torch.ones(32, device="cuda", dtype=torch.float64))
    no(ValueError, wq=torch.ones(31, device="cuda"))
    no(TypeError, positions=pos.long())
    no(ValueError, positions=pos[:3])
    no(ValueError, positions=None)
    no(ValueError, freq_axes=torch.zeros(15, dtype=torch.int32, device="cuda"))
    no(ValueError, q_out=x[:3])
    no(ValueError, k_out=x)
    no(TypeError, q_out=x.clone(), out_dtype=torch.bfloat16)
    no(TypeError, out_dtype=torch.float16)
    no(ValueError, q_out=x.as_strided((4, 2, 32), (32, 128, 1)))
    for kw in (dict(fr=on_gpu(freqs(34), np.float32)), dict(eps=-1.0), dict(eps=float("nan"))):
        no(sa.SAError, **kw)
    big = torch.randn((1, 1, 264), device="cuda")
    no(sa.SAError, q=big, positions=pos[:1].contiguous())
    cu = np.array([0, 2, 5])
    no(sa.SAError, positions=None, cu_seqlens_q_host=cu, cu_seqlens_q=on_gpu(cu, np.int64),
       used_kv_lens=on_gpu([5, 5], np.int32))
    empty, none = sa.sa_norm_rope(x[:0], None, None, None, f, positions=pos[:0])
    assert empty.shape == (0, 2, 32) and none is None


def test_several_axes_need_freq_axes():
    """Without them every pair would be turned by the first axis, and nobody asked for that."""
    x = torch.randn((4, 2, 32), device="cuda")
    f = on_gpu(freqs(32), np.float32)
    pos = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    for kw in (dict(), dict(q_out=torch.empty_like(x))):
        with pytest.raises(ValueError, match="freq_axes"):
            sa.sa_norm_rope(x, None, None, None, f, positions=pos, **kw)
    # one axis, however it is written, and no rotation at all
    a, _ = sa.sa_norm_rope(x, None, None, None, f, positions=pos[:1])
    b, _ = sa.sa_norm_rope(x, None, None, None, f, positions=pos[0].contiguous())
    assert torch.equal(a, b)
    a, _ = sa.sa_norm_rope(x, None, None, None, None, positions=pos)
    assert torch.equal(a, x)
