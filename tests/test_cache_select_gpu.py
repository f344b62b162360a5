"""sa_store_kv, sa_block_bounds and sa_select_blocks against plain 64-bit
statements of their definitions.

Stored codes, scales and bounds are exact by definition (power-of-two scales,
one rounding to nearest even, minima and maxima), so they are compared for
equality; so is the selection, whose reference scores are 64-bit sums."""
import math

import numpy as np
import pytest
import torch

import block_sparse_paged_csr_gb300 as sa

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
         "int8": torch.int8}
QMAX = {"e4m3": 448.0, "int8": 127.0}


def nearest_code(y, kind):
    """Round-to-nearest-even codes (as values) of float64 y inside the range."""
    if kind == "int8":
        return np.round(y)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.abs(y)))
        step = 2.0 ** (np.maximum(e, -6.0) - 3.0)
        return np.where(y == 0, 0.0, np.round(y / step) * step)


def store_reference(x, pages, scales, bt, cu, lens, kind):
    """The definition, page by page.  ``pages`` holds values (codes for the
    8-bit types) in float64, changed in place like ``scales``."""
    ps = pages.shape[2]
    for b, lk in enumerate(lens):
        qo = int(cu[b + 1] - cu[b])
        lk = max(int(lk), 0)
        p0 = lk - qo if lk >= qo else 0
        at = p0
        while at < lk:
            end = min((at // ps + 1) * ps, lk)
            pg = at // ps
            page = bt[b, pg] if pg < bt.shape[1] else -1
            if 0 <= page < pages.shape[0]:
                new = x[cu[b] + at - p0:cu[b] + end - p0].transpose(1, 0, 2)   # [hkv, n, d]
                r0 = at % ps
                if kind in QMAX:
                    for h in range(pages.shape[1]):
                        fin = np.abs(new[h][np.isfinite(new[h])])
                        amax = fin.max() if fin.size else 0.0
                        need = 0.0
                        if amax > 0:
                            need = max(2.0 ** math.ceil(math.log2(amax / QMAX[kind])), 2.0 ** -126)
                        was = scales[page, h] if r0 else 0.0
                        if not (was > 0 and np.isfinite(was)):
                            was = 0.0
                        now = max(was, need)
                        if r0 and now > was:
                            ratio = np.float32(was) / np.float32(now)
                            pages[page, h, :r0] = nearest_code(pages[page, h, :r0] * float(ratio), kind)
                        y = new[h] / now if now > 0 else np.where(np.isnan(new[h]), new[h], 0.0)
                        y = np.clip(y, -QMAX[kind], QMAX[kind])
                        if kind == "int8":
                            y = np.where(np.isnan(y), 0.0, y)
                        pages[page, h, r0:r0 + end - at] = nearest_code(y, kind)
                        scales[page, h] = now
                else:
                    pages[page, :, r0:r0 + end - at] = new
            at = end


def tables(lens, per, rng, extra=0, cols=None):
    live = [max(-(-max(int(n), 0) // per), 0) for n in lens]
    cols = max(max(live), 1) if cols is None else cols
    pool = sum(live) + extra
    perm = rng.permutation(pool).astype(np.int32)
    t = np.full((len(lens), cols), -1, np.int32)
    at = 0
    for b, n in enumerate(live):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, max(pool, 1)


def make_pool(n, hkv, ps, d, kind, rng):
    """Random page contents and scales on the host (values), and on the device."""
    x = rng.standard_normal((n, hkv, ps, d))
    if kind == "int8":
        x = np.clip(np.round(x * 40), -127, 127)
    elif kind == "e4m3":
        x = nearest_code(np.clip(x * 100, -448, 448), kind)
    t = torch.from_numpy(x).cuda().to(TORCH[kind])
    x = t.double().cpu().numpy() if kind != "e4m3" else t.float().double().cpu().numpy()
    s = 2.0 ** rng.integers(-9, -3, (n, hkv)).astype(np.float64)
    return x, s, t, torch.from_numpy(s.astype(np.float32)).cuda()


def host(t):
    return t.float().double().cpu().numpy() if t.dtype == torch.float8_e4m3fn else t.double().cpu().numpy()


def cuda_i(a, dt):
    return torch.from_numpy(np.asarray(a, dt)).cuda()


def run_store(kind, src, qo, lens, hkv, d, ps, seed=0, scale=1.0, edit=None, strided=True,
              extra_rows=3, streams=None):
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(qo)]).astype(np.int64)
    tq = int(cu[-1])
    bt, n = tables(lens, ps, rng, extra=extra_rows)
    kh, ks, kp, ksd = make_pool(n, hkv, ps, d, kind, rng)
    vh, vs, vp, vsd = make_pool(n, hkv, ps, d, kind, rng)
    wide = hkv * 2 + (3 if strided else 0)
    qkv = torch.from_numpy(rng.standard_normal((tq, wide, d)) * scale).cuda()
    if edit is not None:
        edit(qkv)
    qkv = qkv.to(TORCH[src])
    k, v = qkv[:, wide - 2 * hkv:wide - hkv], qkv[:, wide - hkv:]
    kx, vx = k.double().cpu().numpy(), v.double().cpu().numpy()
    if kind == "bf16":     # one rounding on the way in
        kx = k.to(torch.bfloat16).double().cpu().numpy()
        vx = v.to(torch.bfloat16).double().cpu().numpy()
    store_reference(kx, kh, ks, bt, cu, lens, kind)
    store_reference(vx, vh, vs, bt, cu, lens, kind)
    eight = kind in QMAX
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    for _ in range(2):     # the same call again finds its own pages and leaves them
        sa.sa_store_kv(k, v, kp, vp, cuda_i(bt, np.int32), cu, cuda_i(cu, np.int64),
                       cuda_i(lens, np.int32), k_scales=ksd if eight else None,
                       v_scales=vsd if eight else None, status=status)
    assert int(status) == 0
    for got, ref in ((kp, kh), (vp, vh)):
        np.testing.assert_array_equal(host(got), ref)
    if eight:
        np.testing.assert_array_equal(host(ksd), ks)
        np.testing.assert_array_equal(host(vsd), vs)


@pytest.mark.parametrize("kind", ["e4m3", "int8", "bf16", "f32"])
@pytest.mark.parametrize("src", ["f32", "bf16"])
def test_store_ragged(kind, src):
    """Single tokens, page ends inside and at the chunk's ends, a sequence
    without new tokens, one that is new from position 0."""
    run_store(kind, src, [1, 5, 0, 33, 16, 1, 64], [16, 21, 7, 33, 48, 100, 70], 3, 64, 16, seed=1)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("d,ps,qo", [(16, 16, 1), (128, 16, 1), (256, 8, 3), (128, 64, 200),
                                     (256, 256, 300), (48, 12, 30), (128, 128, 129)])
def test_store_sizes(kind, d, ps, qo):
    """Both work splits (a warp or a CTA per page), pages larger than the
    registers hold, sizes that are no powers of two."""
    run_store(kind, "bf16" if d % 32 else "f32", [qo, qo, 1], [qo, qo + 5, 40], 2, d, ps, seed=2)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("scale", [1e-30, 1e-3, 50.0, 1e30])
def test_store_scale_range(kind, scale):
    """New rows far below the page's scale (it stays) and far above (the old
    rows are rounded to the new one)."""
    run_store(kind, "f32", [2, 1, 7], [18, 30, 7], 2, 32, 16, seed=3, scale=scale)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_store_special_values(kind):
    def edit(x):
        x[0] = 0.0                       # a whole token of zeros
        x[1, :, 3] = math.inf
        x[2, :, 4] = -math.inf
        x[3, :, 5] = math.nan
        x[4] = 0.0
        x[4, :, 0] = math.nan            # no finite magnitude but 0
        x[5] *= 1e-42                    # subnormal
        x[6] = 0.0
        x[6, :, 0] = QMAX[kind]          # at the range's end, and one step above
        x[6, :, 1] = -QMAX[kind]
        x[7, :, 0] = float(np.nextafter(np.float32(QMAX[kind]), np.float32(1e9)))
    run_store(kind, "f32", [1] * 8, [1, 1, 17, 17, 17, 1, 17, 33], 2, 32, 16, seed=4, edit=edit)


def test_store_scale_of_a_callers_own():
    """A page whose scale is no power of two keeps it while it suffices: codes
    are x / s to the nearest; garbage scales count as none."""
    ps, d = 16, 32
    bt = np.array([[0], [1], [2]], np.int32)
    kp = torch.zeros((3, 1, ps, d), dtype=torch.int8, device="cuda")
    kp[:, :, :4] = 100
    ks = torch.tensor([[0.3], [math.nan], [-1.0]], device="cuda")
    vp, vs = kp.clone(), ks.clone()
    x = torch.linspace(-9, 9, 3 * d, device="cuda").view(3, 1, d)
    cu = np.arange(4)
    lens = np.full(3, 5)
    sa.sa_store_kv(x, x, kp, vp, cuda_i(bt, np.int32), cu, cuda_i(cu, np.int64),
                   cuda_i(lens, np.int32), k_scales=ks, v_scales=vs)
    assert ks[0, 0] == torch.tensor(0.3)
    q = x[0, 0].cpu().numpy() / np.float32(0.3)
    np.testing.assert_array_equal(kp[0, 0, 4].cpu().numpy(), np.round(q).astype(np.int8))
    assert (kp[0, 0, :4] == 100).all()
    for b in (1, 2):                      # the old rows stood for nothing
        amax = float(x[b].abs().max())
        assert float(ks[b, 0]) == 2.0 ** math.ceil(math.log2(amax / 127))
        assert (kp[b, 0, :4] == 0).all()
    assert torch.equal(kp, vp)


def test_store_lengths_and_tables():
    """Shorter than its new tokens, empty, dropped pages, ids past the pool,
    positions past the table."""
    hkv, d, ps = 2, 32, 16
    qo, lens = [40, 3, 20, 20, 40], [20, 0, 40, 40, 100]
    cu = np.concatenate([[0], np.cumsum(qo)]).astype(np.int64)
    rng = np.random.default_rng(5)
    bt = np.array([[0, 1, 2], [3, 3, 3], [4, -1, 5], [6, 99, 7], [8, 9, 10]], np.int32)
    kh, ks, kp, ksd = make_pool(12, hkv, ps, d, "int8", rng)
    vh, vs, vp, vsd = make_pool(12, hkv, ps, d, "int8", rng)
    k = torch.randn((int(cu[-1]), hkv, d), device="cuda")
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    args = (cuda_i(bt, np.int32), cu, cuda_i(cu, np.int64), cuda_i(lens, np.int32))
    sa.sa_store_kv(k, k, kp, vp, *args, k_scales=ksd, v_scales=vsd, status=status)
    assert sa.sa_status_string(int(status)) == "shape mismatch"
    x = k.double().cpu().numpy()
    store_reference(x, kh, ks, bt, cu, lens, "int8")
    store_reference(x, vh, vs, bt, cu, lens, "int8")
    np.testing.assert_array_equal(host(kp), kh)
    np.testing.assert_array_equal(host(vp), vh)
    np.testing.assert_array_equal(host(ksd), ks)
    # without a status word the call works the same
    sa.sa_store_kv(k, k, kp, vp, *args, k_scales=ksd, v_scales=vsd)
    np.testing.assert_array_equal(host(kp), kh)


def test_store_far_pages():
    """Offsets past 2^31 elements: the last pages of a 2.6 G element pool."""
    hkv, d, ps = 2, 128, 64
    n = 160000
    kp = torch.zeros((n, hkv, ps, d), dtype=torch.int8, device="cuda")
    vp = torch.zeros((n, hkv, ps, d), dtype=torch.int8, device="cuda")
    ks = torch.zeros((n, hkv), device="cuda")
    vs = torch.zeros((n, hkv), device="cuda")
    bt = np.array([[n - 1, n - 2]], np.int32)
    cu = np.array([0, 70], np.int64)
    x = torch.randn((70, hkv, d), device="cuda")
    y = torch.randn((70, hkv, d), device="cuda")
    a = (cuda_i(bt, np.int32), cu, cuda_i(cu, np.int64), cuda_i([70], np.int32))
    sa.sa_store_kv(x, y, kp, vp, *a, k_scales=ks, v_scales=vs)
    for t, pages, scales in ((x, kp, ks), (y, vp, vs)):
        got = pages[n - 1].float() * scales[n - 1][:, None, None]
        ref = t[:64].transpose(0, 1)
        # half a step of the page's scale
        assert ((got - ref).abs() <= 0.5 * scales[n - 1][:, None, None]).all()
        assert (pages[n - 2, :, 6:] == 0).all() and (pages[n - 2, :, :6] != 0).any()
        assert (pages[:n - 2] == 0).all()
    bounds = torch.zeros((2, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    sa.sa_block_bounds(kp, *a, bounds, cuda_i([[1]], np.int32), 128, k_scales=ks)
    vals = torch.cat([kp[n - 1].float() * ks[n - 1][:, None, None],
                      (kp[n - 2].float() * ks[n - 2][:, None, None])[:, :6]], 1)
    assert torch.equal(bounds[1, :, 0].float(), vals.amin(1))
    assert torch.equal(bounds[1, :, 1].float(), vals.amax(1))


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_store_leaves_pages_without_new_rows(kind):
    """A sequence without new tokens whose length ends inside a page: the page
    and its scale stay as they are, whatever the scale (0.3, negative, NaN)."""
    hkv, d, ps = 2, 32, 16
    lens, qo = [7, 23, 5, 9], [0, 0, 0, 1]
    cu = np.concatenate([[0], np.cumsum(qo)]).astype(np.int64)
    bt = np.array([[0, -1], [1, 2], [3, -1], [4, -1]], np.int32)
    kp = torch.full((5, hkv, ps, d), 3, dtype=torch.uint8, device="cuda").view(TORCH[kind])
    ks = torch.tensor([[-2.0, 0.3], [1.0, 1.0], [-0.5, math.nan], [math.inf, 0.0], [0.25, 0.25]],
                      device="cuda")
    vp, vs = kp.clone(), -ks
    before = [t.clone() for t in (kp, vp, ks, vs)]
    x = torch.ones((1, hkv, d), device="cuda")
    sa.sa_store_kv(x, x, kp, vp, cuda_i(bt, np.int32), cu, cuda_i(cu, np.int64),
                   cuda_i(lens, np.int32), k_scales=ks, v_scales=vs)
    for t, was in zip((kp, vp, ks, vs), before):
        np.testing.assert_array_equal(t[:4].cpu().view(torch.uint8).numpy(),
                                      was[:4].cpu().view(torch.uint8).numpy())


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_store_page_shared_with_an_idle_sequence(kind):
    """Two sequences over one partly filled page, of which one appends a larger
    row: the page takes the larger scale (many pairs, so that the two meet)."""
    hkv, d, ps, n = 8, 64, 16, 300
    order = np.random.default_rng(1).permutation(2 * n)
    lens, qo = np.zeros(2 * n, np.int64), np.zeros(2 * n, np.int64)
    bt = np.zeros((2 * n, 1), np.int32)
    for i, s in enumerate(order):          # i < n: appends to page i; else idle on page i - n
        lens[s], qo[s], bt[s, 0] = (8, 1, i) if i < n else (7, 0, i - n)
    cu = np.concatenate([[0], np.cumsum(qo)]).astype(np.int64)
    unit = 2.0 ** -6
    for _ in range(5):
        kp = torch.ones((n, hkv, ps, d), device="cuda").mul_(64).to(TORCH[kind])
        ks = torch.full((n, hkv), unit, device="cuda")
        vp, vs = kp.clone(), ks.clone()
        x = torch.full((n, hkv, d), 64.0 * 16 * unit, device="cuda")
        sa.sa_store_kv(x, x, kp, vp, cuda_i(bt, np.int32), cu, cuda_i(cu, np.int64),
                       cuda_i(lens, np.int32), k_scales=ks, v_scales=vs)
        for pages, scales in ((kp, ks), (vp, vs)):
            v = pages.float() * scales[:, :, None, None]
            assert (v[:, :, :7] == 64 * unit).all() and (v[:, :, 7] == 64 * 16 * unit).all()


# ----------------------------------------------------------------------------- bounds

def outward(x, up):
    """float64 -> the bf16 value (as float64) at or beyond it."""
    f = np.asarray(x, np.float32)
    bits = f.view(np.uint32).astype(np.uint64)
    rest = (bits & 0xFFFF) != 0
    away = rest & ((bits >> 31 == 0) if up else (bits >> 31 == 1))
    out = (((bits >> 16) + away) << 16).astype(np.uint32).view(np.float32)
    return out.astype(np.float64)


@pytest.mark.parametrize("kind", ["e4m3", "int8", "bf16", "f32"])
@pytest.mark.parametrize("hkv,d,ps,bs", [(2, 32, 16, 32), (1, 128, 16, 64), (3, 64, 8, 128),
                                         (1, 256, 32, 32), (2, 48, 12, 36), (1, 16, 4, 16),
                                         (2, 48, 32, 64), (1, 128, 64, 128)])
def test_bounds(kind, hkv, d, ps, bs):
    rng = np.random.default_rng(6)
    qo = [1, 0, 70, 5, 1, 200]
    lens = [50, 60, 70, 65, 64, 201]
    cu = np.concatenate([[0], np.cumsum(qo)]).astype(np.int64)
    bt, n = tables(lens, ps, rng)
    per = bs // ps
    cols = -(-bt.shape[1] // per)
    bt = np.concatenate([bt, np.full((len(lens), cols * per - bt.shape[1]), -1, np.int32)], 1)
    kh, ks, kp, ksd = make_pool(n, hkv, ps, d, kind, rng)
    if kind in ("e4m3", "bf16", "f32"):
        kp.view(-1)[5::97] = math.nan
        kh.reshape(-1)[5::97] = math.nan
    bt[2, 0] = -1                       # a dropped page inside a block
    rows, nb = tables(lens, bs, rng, extra=2, cols=cols)
    rows[5, 0] = -1                     # a block the caller keeps no bounds for
    out = torch.full((nb, hkv, 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ref = np.full((nb, hkv, 2, d), 7.0)
    if kind in QMAX:
        kh = kh * ks[:, :, None, None]
    for b, lk in enumerate(lens):
        for j in range((lk - qo[b]) // bs, -(-lk // bs)):
            if qo[b] == 0 or rows[b, j] < 0:
                continue
            keys = [kh[bt[b, p // ps], :, p % ps] for p in range(j * bs, min((j + 1) * bs, lk))
                    if bt[b, p // ps] >= 0]
            k = np.stack(keys, 1) if keys else np.zeros((hkv, 0, d))
            nan = np.isnan(k)
            ref[rows[b, j], :, 0] = outward(np.where(nan, np.inf, k).min(1, initial=np.inf), False)
            ref[rows[b, j], :, 1] = outward(np.where(nan, -np.inf, k).max(1, initial=-np.inf), True)
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    got = sa.sa_block_bounds(kp, cuda_i(bt, np.int32), cu, cuda_i(cu, np.int64),
                             cuda_i(lens, np.int32), out, cuda_i(rows, np.int32), bs,
                             k_scales=ksd if kind in QMAX else None, status=status)
    assert got is out and int(status) == 0
    np.testing.assert_array_equal(host(out), ref)


def test_bounds_without_keys_and_bad_ids():
    """All pages dropped: (+inf, -inf).  A row past the pool and a page past
    the cache are reported and touch nothing."""
    kp = torch.zeros((4, 1, 16, 16), dtype=torch.bfloat16, device="cuda")
    cu = np.array([0, 64], np.int64)
    out = torch.zeros((3, 1, 2, 16), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int64, device="cuda")

    def call(bt, rows):
        status.zero_()
        sa.sa_block_bounds(kp, cuda_i(bt, np.int32), cu, cuda_i(cu, np.int64),
                           cuda_i([64], np.int32), out, cuda_i(rows, np.int32), 32, status=status)
        return int(status)

    assert call([[-1, -1, 0, 1]], [[0, 1]]) == 0
    assert (out[0, 0, 0] == math.inf).all() and (out[0, 0, 1] == -math.inf).all()
    assert (out[1] == 0).all()
    assert sa.sa_status_string(call([[0, 1, 2, 3]], [[2, 9]])) == "shape mismatch"
    assert (out[2] == 0).all()
    assert sa.sa_status_string(call([[9, 1, 2, 3]], [[2, 1]])) == "shape mismatch"


def outward64(x, up):
    """float64 -> the nearest bf16 value (as float64) at or beyond it."""
    m, e = np.frexp(np.asarray(x, np.float64))
    m = (np.ceil if up else np.floor)(m * 256.0)
    return np.ldexp(m, e - 8)


@pytest.mark.parametrize("ps,bs,d", [(16, 32, 32), (4, 16, 64), (64, 128, 128)])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("scales", ["negative", "signs", "any"])
def test_bounds_scales_of_any_sign(kind, scales, ps, bs, d):
    """Scales of a caller's own: negative ones turn smallest and largest round."""
    rng = np.random.default_rng(8)
    hkv, lens, qo = 2, [3 * bs + 5, bs, 2 * bs - 1], [3 * bs + 5, 2, bs]
    cu = np.concatenate([[0], np.cumsum(qo)]).astype(np.int64)
    bt, n = tables(lens, ps, rng)
    cols = -(-bt.shape[1] * ps // bs)
    bt = np.concatenate([bt, np.full((len(lens), cols * bs // ps - bt.shape[1]), -1, np.int32)], 1)
    kh, _, kp, _ = make_pool(n, hkv, ps, d, kind, rng)
    if scales == "negative":
        s = -(2.0 ** rng.integers(-9, -3, (n, hkv)))
    elif scales == "signs":
        s = 2.0 ** rng.integers(-9, -3, (n, hkv)) * rng.choice([-1.0, 0.0, 1.0], (n, hkv))
    else:
        s = rng.uniform(-0.1, 0.1, (n, hkv))
    s = s.astype(np.float32)
    rows, nb = tables(lens, bs, rng, cols=cols)
    out = torch.zeros((nb, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    sa.sa_block_bounds(kp, cuda_i(bt, np.int32), cu, cuda_i(cu, np.int64), cuda_i(lens, np.int32),
                       out, cuda_i(rows, np.int32), bs, k_scales=torch.from_numpy(s).cuda())
    vals = kh * s.astype(np.float64)[:, :, None, None]
    got = host(out)
    for b, lk in enumerate(lens):
        for j in range((lk - qo[b]) // bs, -(-lk // bs)):
            k = np.stack([vals[bt[b, p // ps], :, p % ps] for p in range(j * bs, min((j + 1) * bs, lk))], 1)
            lo, hi = got[rows[b, j], :, 0], got[rows[b, j], :, 1]
            np.testing.assert_array_equal(lo, outward64(k.min(1), False))
            np.testing.assert_array_equal(hi, outward64(k.max(1), True))


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_bounds_enclose_the_exact_keys(kind):
    """Products that lie just beside a bf16 number, where f32 would round to it:
    the bounds enclose the exact product."""
    codes = [c for c in range(1, 100 if kind == "int8" else 16)]
    n, d = 2 * len(codes), 32
    c = np.array(codes * 2, np.float32) * np.repeat([1, -1], len(codes)).astype(np.float32)
    s = np.float32(1) / np.abs(c)
    kp = torch.from_numpy(c).cuda()[:, None, None, None].expand(n, 1, 16, d).contiguous().to(TORCH[kind])
    bt = np.arange(n, dtype=np.int32)[:, None]
    cu = np.arange(n + 1, dtype=np.int64) * 16
    out = torch.zeros((n, 1, 2, d), dtype=torch.bfloat16, device="cuda")
    sa.sa_block_bounds(kp, cuda_i(bt, np.int32), cu, cuda_i(cu, np.int64),
                       cuda_i(np.full(n, 16), np.int32), out, cuda_i(bt, np.int32), 16,
                       k_scales=torch.from_numpy(s)[:, None].cuda())
    exact = c.astype(np.float64) * s.astype(np.float64)
    assert (exact != np.float32(exact)).any()              # (some are not f32 numbers)
    for x, up in ((0, False), (1, True)):
        np.testing.assert_array_equal(host(out)[:, 0, x], np.repeat(outward64(exact, up)[:, None], d, 1))


# ----------------------------------------------------------------------------- selection

def visible(cu, lens, causal, bs, msb):
    """(sequence, blocks in sight) of every query."""
    out = []
    for b, lk in enumerate(lens):
        qo, lk = int(cu[b + 1] - cu[b]), max(int(lk), 0)
        for t in range(qo):
            seen = lk
            if causal:
                pos = t if causal == 2 or lk < qo else lk - qo + t
                seen = min(lk, pos + 1)
            out.append((b, min(-(-seen // bs), msb)))
    return out


def select_reference(q, bounds, rows, cu, lens, bs, topk, causal, sink=0, local=0):
    tq, hq, d = q.shape
    hkv = bounds.shape[1]
    out = np.full((tq, hkv, topk), -1, np.int32)
    with np.errstate(invalid="ignore", over="ignore"):
        for i, (b, n) in enumerate(visible(cu, lens, causal, bs, rows.shape[1])):
            g = hq // hkv
            for h in range(hkv):
                ids = np.array([j for j in range(n) if 0 <= rows[b, j] < bounds.shape[0]
                                and not bounds[rows[b, j], h, 0, 0] > bounds[rows[b, j], h, 1, 0]],
                               np.int64)
                if not len(ids):
                    continue
                x = q[i, h * g:(h + 1) * g]                                    # [g, d]
                neg = np.where(np.isnan(x), x, np.minimum(x, 0)).sum(0)
                pos = np.where(np.isnan(x), x, np.maximum(x, 0)).sum(0)
                box = bounds[rows[b, ids], h]                                  # [n, 2, d]
                s = (box[:, 0] * neg).sum(1) + (box[:, 1] * pos).sum(1)
                # ranks: forced, numbers from the largest, NaN; then the id
                cls = np.where((ids < sink) | (ids >= n - local), 0, np.where(np.isnan(s), 2, 1))
                s = np.where(cls == 1, s, 0.0)
                order = np.lexsort((ids, -s, cls))[:topk]
                pick = np.sort(ids[order])
                out[i, h, :len(pick)] = pick
    return out


def run_select(q, bounds, rows, cu, lens, bs, topk, causal=1, sink=0, local=0, ref=None,
               expect=0, **kw):
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    got = sa.sa_select_blocks(q, bounds, cuda_i(rows, np.int32), cu, cuda_i(cu, np.int64),
                              cuda_i(lens, np.int32), bs, topk, causal, sink, local,
                              status=status, **kw)
    assert int(status) == expect
    if ref is None:
        ref = select_reference(q.double().cpu().numpy(), bounds.double().cpu().numpy(), rows, cu,
                               lens, bs, topk, causal, sink, local)
    got = got.cpu().numpy()
    bad = np.argwhere(got != ref)
    assert not len(bad), f"{len(bad)} ids differ, first at {bad[0]}: {got[tuple(bad[0][:2])]} " \
                         f"vs {ref[tuple(bad[0][:2])]}"
    return got


def make_bounds(n, hkv, d, gen, width=1.0):
    mid = torch.randn((n, hkv, 1, d), generator=gen, device="cuda")
    half = width * torch.rand((n, hkv, 1, d), generator=gen, device="cuda")
    return torch.cat([mid - half, mid + half], 2).to(torch.bfloat16)


def problem(qo, lens, hq, hkv, d, bs, act="f32", seed=0, width=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(qo)]).astype(np.int64)
    rows, n = tables(lens, bs, rng)
    q = torch.randn((int(cu[-1]), hq, d), generator=gen, device="cuda").to(TORCH[act])
    return q, make_bounds(n, hkv, d, gen, width), rows, cu, np.asarray(lens)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("causal", [0, 1, 2])
@pytest.mark.parametrize("d,g", [(8, 1), (16, 3), (32, 2), (48, 5), (64, 4), (128, 8), (192, 1),
                                 (256, 7)])
def test_select_ragged(act, causal, d, g):
    """Single queries and chunks, sequences without queries or keys, shorter
    than their queries, lengths at and past block borders."""
    p = problem([1, 4, 0, 9, 3, 2], [700, 321, 50, 1600, 0, 1], 2 * g, 2, d, 32, act, seed=d + g)
    run_select(*p, 32, 7, causal)


@pytest.mark.parametrize("topk", [1, 2, 31, 33, 64, 200])
def test_select_topk(topk):
    p = problem([2, 1, 3], [2000, 900, 1030], 4, 2, 64, 16, seed=topk)
    run_select(*p, 16, topk)


@pytest.mark.parametrize("sink,local", [(1, 0), (0, 2), (2, 3), (4, 4), (8, 0)])
def test_select_forced(sink, local):
    p = problem([3, 1, 2], [2000, 90, 17], 4, 2, 64, 16, seed=9)
    got = run_select(*p, 16, 8, 1, sink, local)
    assert (got[0, :, :sink] == np.arange(sink)).all()


@pytest.mark.parametrize("n", [255, 256, 257, 1000, 2047, 4100, 16384])
def test_select_many_blocks(n):
    p = problem([1, 2], [n * 16, n * 16 - 40], 8, 2, 32, 16, seed=n)
    run_select(*p, 16, 64)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("d", [8, 32, 64, 128, 256])
def test_select_many_sequences(d, act):
    """More (sequence, head, 256 blocks) units than are resident at a time, an
    odd number of them per row, single queries."""
    lens = [(700 * 16 - 37 * i) if i % 7 else 5 * i for i in range(90)]
    p = problem([1] * 90, lens, 4, 2, d, 16, act, seed=d + 1)
    run_select(*p, 16, 33)


def test_select_missing_blocks_and_bad_rows():
    q, bounds, rows, cu, lens = problem([2, 1], [1600, 800], 4, 2, 64, 16, seed=11)
    rows[0, ::3] = -1
    bounds[rows[0, 1], :, 0] = math.inf          # a block without keys
    bounds[rows[0, 1], :, 1] = -math.inf
    bounds[rows[0, 4], 1, 0] = math.inf          # ... for one of the heads
    bounds[rows[0, 4], 1, 1] = -math.inf
    run_select(q, bounds, rows, cu, lens, 16, 12)
    run_select(q, bounds, rows, cu, lens, 16, 60)       # fewer candidates than asked for
    run_select(q, bounds, rows, cu, lens, 16, 128)      # ... than blocks in sight
    run_select(q, bounds, rows, cu, lens, 16, 12, 1, 2, 2)   # a forced block that is not there
    rows[1, 5] = len(bounds) + 3
    run_select(q, bounds, rows, cu, lens, 16, 12, expect=4)
    run_select(q, bounds, rows, cu, lens, 16, 80, expect=4)


def test_select_ties():
    """Equal scores: the lower block; zero queries: the first blocks."""
    q, bounds, rows, cu, lens = problem([2, 1, 2], [3200, 1600, 3200], 4, 2, 64, 16, seed=12)
    rows[0, :] = np.arange(rows.shape[1]) % 7            # every block seven-fold and more
    q[3] = 0.0
    run_select(q, bounds, rows, cu, lens, 16, 20)
    run_select(q, bounds, rows, cu, lens, 16, 20, 1, 1, 3)
    bounds[:] = bounds[:1]                                # all alike
    run_select(q, bounds, rows, cu, lens, 16, 33)


def test_select_needs_more_than_f32():
    """Scores of one size that differ far below f32's reach: a common part of
    2^20 and differences of 2^-20 and up.  All products and sums of the
    reference are exact in 64 bits."""
    d, n, bs, topk = 64, 300, 16, 40
    rng = np.random.default_rng(13)
    q = torch.ones((2, 2, d), device="cuda")
    q[:, :, 1] = 2.0 ** -20
    q[1, :, 2] = -2.0 ** -19
    bounds = torch.zeros((n, 1, 2, d), dtype=torch.bfloat16, device="cuda")
    bounds[:, :, :, 0] = 2.0 ** 20
    small = torch.from_numpy(rng.permutation(n).astype(np.float32)).cuda()
    # up to 299 needs 9 bits: split over two channels of bf16
    bounds[:, 0, :, 1] = (small // 2).to(torch.bfloat16)[:, None]
    bounds[:, 0, :, 2] = 0.0
    bounds[:, 0, 1, 3] = ((small % 2) * 2.0 ** -21).to(torch.bfloat16)
    rows = np.arange(n, dtype=np.int32)[None]
    cu = np.array([0, 2])
    got = run_select(q, bounds, rows, cu, np.array([n * bs]), bs, topk, 0)
    order = torch.sort(small.cpu(), descending=True).indices[:topk].sort().values.numpy()
    assert (got[0, 0] == order).all()


def test_select_border_in_many_rows():
    """Random scores with a border that f32 leaves open in many rows: bounds in
    a narrow band on a large common offset."""
    q, bounds, rows, cu, lens = problem([40, 30], [8000, 8000], 8, 2, 128, 16, seed=14)
    centre = torch.randn((1, 2, 2, 128), device="cuda") * 64
    step = torch.randint(0, 2, bounds.shape, device="cuda") * 0.5
    bounds = (centre.sort(2).values.round() + step).to(torch.bfloat16)[..., :]
    bounds = bounds.expand(len(bounds), 2, 2, 128).contiguous()
    run_select(q, bounds, rows, cu, lens, 16, 50)


def test_select_not_finite():
    q, bounds, rows, cu, lens = problem([5], [1600], 4, 2, 32, 16, seed=15)
    q[0, 0, 3] = math.nan                      # every score of a head NaN: the first blocks
    q[1, 2, 4] = math.inf
    q[2, 1, 5] = -math.inf
    bounds[rows[0, 7], 0, 1, 9] = math.inf     # a key of infinite size
    bounds[rows[0, 8], 1, 0, 9] = -math.inf
    bounds[rows[0, 9], 1, 1, 3] = math.nan
    run_select(q, bounds, rows, cu, lens, 16, 9)
    run_select(q, bounds, rows, cu, lens, 16, 9, 1, 1, 2)
    q2 = torch.randn_like(q) * 1e30            # sums past f32
    b2 = (bounds.float().nan_to_num(0, 0, 0) * 1e30).to(torch.bfloat16)
    run_select(q2, b2, rows, cu, lens, 16, 9)


@pytest.mark.parametrize("d", [8, 32, 64, 128, 256])
@pytest.mark.parametrize("qo", [1, 3, 40])
@pytest.mark.parametrize("topk", [5, 90])
def test_select_leaves_out_rows_of_no_block(qo, d, topk):
    """A bounds row with lo[0] > hi[0] is no block, finite or not, however high
    its score: with more blocks in sight than are taken and with fewer."""
    q, bounds, rows, cu, lens = problem([qo, 1], [1600, 900], 4, 2, d, 16, seed=31 + d)
    gen = np.random.default_rng(d)
    for b in range(2):
        n = -(-int(lens[b]) // 16)
        for j in gen.permutation(n)[:n // 5]:
            r, h = rows[b, j], int(gen.integers(2))
            bounds[r, h, 0] = -50.0                    # wide, so high scores ..
            bounds[r, h, 1] = 50.0
            bounds[r, h, 0, 0] = 2.0 ** -7             # .. but for channel 0
            bounds[r, h, 1, 0] = -2.0 ** -7
    got = run_select(q, bounds, rows, cu, lens, 16, topk)
    box = bounds.float().cpu().numpy()
    seq = np.searchsorted(cu, np.arange(len(got)), side="right") - 1
    for i in range(len(got)):
        for h in range(2):
            ids = got[i, h][got[i, h] >= 0]
            assert (box[rows[seq[i], ids], h, 0, 0] <= box[rows[seq[i], ids], h, 1, 0]).all()


@pytest.mark.parametrize("qo", [1, 4, 16])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("big", [1.0, 1.9921875, -1.0])
def test_select_small_terms_beside_large_ones(qo, d, big):
    """Scores whose small terms a sum cuts off beside two large ones: half of
    the blocks have all of them positive, the other half all of them negative
    and one more term, smaller than the difference, that the sum keeps.  Which
    half comes first turns on what was cut off.  Small terms of many sizes; all
    products and all sums in 64 bits are exact."""
    n, bs, topk = 600, 16, 300
    q = torch.ones((qo, 2, d), device="cuda")
    q[:, 1] = -1.0                                     # weights 1 and -1 in every channel
    rng = np.random.default_rng(d)
    rows = rng.permutation(n).astype(np.int32)[None]
    cu = np.array([0, qo])
    lens = np.array([n * bs])
    for k in range(21, 31):
        tiny = 1.9921875 * 2.0 ** -k
        small = [c for c in range(2, d) if c not in (4, 5)]
        for part in (0.3, 0.55, 0.65, 0.75, 0.9):
            first = rng.permutation(n)[:n // 2]        # the half that should come in
            sign = np.full((n, 1), -1.0)
            sign[first] = 1.0
            lo, hi = np.zeros((n, d)), np.zeros((n, d))
            hi[:, small] = sign * tiny
            lo[:, small] = -sign * tiny                # (times -1: the same again)
            lo[:, 1] = lo[:, 4] = -big                 # times -1: among the first terms
            kept = torch.tensor(part * 4 * len(small) * tiny).to(torch.bfloat16).item()
            hi[sign[:, 0] < 0, 5] = kept
            box = np.stack([lo, hi], 1)[:, None]
            bounds = torch.from_numpy(box).to(torch.bfloat16)
            assert torch.equal(bounds.double(), torch.from_numpy(box))
            place = torch.empty_like(bounds)
            place[torch.from_numpy(rows[0]).long()] = bounds
            ref = np.tile(np.sort(first).astype(np.int32), (qo, 1, 1))
            run_select(q, place.cuda(), rows, cu, lens, bs, topk, 0, ref=ref)


def test_select_in_parts():
    """More scores than the workspace holds at a time."""
    qo, n, bs, topk = 1100, 16000, 16, 24
    gen = torch.Generator(device="cuda").manual_seed(16)
    cu = np.array([0, qo])
    lens = np.array([n * bs])
    rows = np.random.default_rng(16).permutation(n).astype(np.int32)[None]
    q = torch.randn((qo, 8, 8), generator=gen, device="cuda")
    bounds = make_bounds(n, 8, 8, gen)
    ws = sa.allocate_select_workspace(qo, 1, 8, 8, n, "cuda")
    assert ws.numel() < qo * 8 * n * 4
    nblk = torch.div(torch.arange(qo, device="cuda") + n * bs - qo, bs, rounding_mode="floor") + 1
    box = bounds[torch.from_numpy(rows[0]).cuda().long()].double()          # [n, hkv, 2, d]
    w = torch.stack([q.double().clamp(max=0), q.double().clamp(min=0)], 2)  # [qo, hkv, 2, d]
    score = torch.einsum("qhsd,nhsd->qhn", w, box)
    col = torch.arange(n, device="cuda")
    score = score.masked_fill(col >= nblk[:, None, None], -math.inf)
    ref = torch.sort(score, dim=2, descending=True, stable=True).indices[:, :, :topk].sort(2).values
    run_select(q, bounds, rows, cu, lens, bs, topk, ref=ref.int().cpu().numpy(), workspace=ws)


def test_select_arguments():
    q, bounds, rows, cu, lens = problem([2], [320], 4, 2, 32, 16, seed=17)
    a = (cu, cuda_i(cu, np.int64), cuda_i(lens, np.int32), 16, 4, True)
    r = cuda_i(rows, np.int32)
    with pytest.raises(ValueError):
        sa.sa_select_blocks(q.transpose(0, 1), bounds, r, *a)
    with pytest.raises(ValueError):
        sa.sa_select_blocks(q, bounds[..., :16], r, *a)
    with pytest.raises(TypeError):
        sa.sa_select_blocks(q, bounds.float(), r, *a)
    with pytest.raises(ValueError):
        sa.sa_select_blocks(q, bounds, r.cpu(), *a)
    with pytest.raises(ValueError):
        sa.sa_select_blocks(q, bounds, r, *a, selected=torch.empty((2, 2, 5), dtype=torch.int32,
                                                                   device="cuda"))
    with pytest.raises(sa.SAError):
        sa.sa_select_blocks(q, bounds, r, *a, workspace=torch.empty(64, dtype=torch.uint8,
                                                                    device="cuda"))
    with pytest.raises(sa.SAError):
        sa.sa_select_blocks(q[:, :3].contiguous(), bounds, r, *a)


def test_on_another_stream_and_in_a_graph():
    """Store, bounds and selection on a stream of the caller's, captured and
    replayed with new contents."""
    hkv, d, ps, bs, topk = 2, 64, 16, 32, 5
    lens = np.array([500, 321, 64])
    cu = np.arange(4)
    rng = np.random.default_rng(18)
    bt, n = tables(np.ceil(lens / bs) * bs, ps, rng)
    rows, nb = tables(lens, bs, rng)
    pool = torch.randint(-99, 99, (n, hkv, ps, d), device="cuda").to(torch.int8)
    start = torch.full((n, hkv), 2.0 ** -6, device="cuda")
    k = torch.randn((3, hkv, d), device="cuda")
    v = torch.randn((3, hkv, d), device="cuda")
    q = torch.randn((3, 4, d), device="cuda")
    full = torch.zeros((nb, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    a = (cuda_i(bt, np.int32), cu, cuda_i(cu, np.int64), cuda_i(lens, np.int32))
    r = cuda_i(rows, np.int32)
    # the bounds of everything stored so far: a call in which all is new
    every = np.concatenate([[0], np.cumsum(lens)])
    sa.sa_block_bounds(pool, a[0], every, cuda_i(every, np.int64), a[3], full, r, bs, k_scales=start)

    def step(kp, vp, ks, vs, bounds, stream=None, **kw):
        sa.sa_store_kv(k, v, kp, vp, *a, k_scales=ks, v_scales=vs, stream=stream)
        sa.sa_block_bounds(kp, *a, bounds, r, bs, k_scales=ks, stream=stream)
        return sa.sa_select_blocks(q, bounds, r, *a[1:], bs, topk, True, stream=stream, **kw)

    def fresh():
        return pool.clone(), pool.clone(), start.clone(), start.clone(), full.clone()

    ref = step(*(want := fresh()))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    state = fresh()
    torch.cuda.synchronize()
    got = step(*state, stream=side)
    side.synchronize()
    assert torch.equal(got, ref)
    for x, y in zip(state, want):
        assert torch.equal(x, y)
    ws = sa.allocate_select_workspace(3, 3, hkv, d, rows.shape[1], "cuda")
    sel = torch.empty((3, hkv, topk), dtype=torch.int32, device="cuda")
    state = fresh()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*state, selected=sel, workspace=ws)
    for seed in range(2):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, device="cuda"))
        for x, y in zip(state, fresh()):
            x.copy_(y)
        ref = step(*(want := fresh()))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(sel, ref)
        for x, y in zip(state, want):
            assert torch.equal(x, y)


def test_prompts_in_a_row_and_in_a_graph():
    """Selection for prompts: calls that follow one another on one workspace
    without a synchronisation, bounds rewritten in between, and a captured call
    replayed with new queries and bounds."""
    hkv, d, bs, topk = 2, 128, 16, 12
    _, bounds, rows, cu, lens = problem([130, 0, 20, 300], [4000, 50, 5200, 9000], 8, hkv, d, bs,
                                        seed=19)
    a = (cuda_i(rows, np.int32), cu, cuda_i(cu, np.int64), cuda_i(lens, np.int32), bs, topk, True)
    gen = torch.Generator(device="cuda").manual_seed(20)
    n = 12
    qs = [torch.randn((int(cu[-1]), 8, d), generator=gen, device="cuda") for _ in range(n)]
    boxes = [make_bounds(bounds.shape[0], hkv, d, gen) for _ in range(n)]
    ref = []
    for q, box in zip(qs, boxes):
        ref.append(sa.sa_select_blocks(q, box, *a))
        torch.cuda.synchronize()
    ws = sa.allocate_select_workspace(int(cu[-1]), 4, hkv, d, rows.shape[1], "cuda")
    box = boxes[0].clone()
    got = []
    for q, new in zip(qs, boxes):
        box.copy_(new)
        got.append(sa.sa_select_blocks(q, box, *a, workspace=ws))
    torch.cuda.synchronize()
    for x, y in zip(got, ref):
        assert torch.equal(x, y)
    assert not torch.equal(ref[0], ref[1])
    q, sel = qs[0].clone(), torch.empty_like(ref[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sa.sa_select_blocks(q, box, *a, workspace=ws, selected=sel)
    for i in range(n):
        q.copy_(qs[i])
        box.copy_(boxes[i])
        g.replay()
        assert torch.equal(sel, ref[i])


@pytest.mark.parametrize("qo,d", [(1, 128), (3, 64), (20, 128), (3, 256)])
def test_selection_waits_run_out(qo, d):
    """Score kernels whose copies never come give up, wait (as long) for those
    that may be in flight, report it and end; the next call is clean."""
    q, bounds, rows, cu, lens = problem([qo, qo], [9000, 4000], 4, 2, d, 16, seed=41)
    a = (q, bounds, cuda_i(rows, np.int32), cu, cuda_i(cu, np.int64), cuda_i(lens, np.int32), 16, 7, 1)
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    sa.sa_debug_stall(sa.STALL_SELECT_COPIES, 2000)
    try:
        sa.sa_select_blocks(*a, status=status)
        torch.cuda.synchronize()
    finally:
        sa.sa_debug_stall(sa.STALL_NONE, 0)
    assert int(status) == 9, sa.sa_status_string(int(status))
    run_select(q, bounds, rows, cu, lens, 16, 7)
