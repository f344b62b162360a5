"""Attention over a cache held in 8 bits (e4m3, int8; a scale per page and kv
head) against the oracle in 64 bits on the values the codes stand for.

Tolerances (row-normalised, as in the other parity tests): the fused decode
and general kernels take codes exactly and split Q and P into two f16 parts or
keep them in f32, so they are held to the f32 class, 1e-4; a bf16 output adds
its rounding of 2^-8; the tensor-core kernel rounds Q, P and K/V to bf16, 2e-2 for keys of unit size.
There the error is that of the scores: rounding q and k moves a score by at most
2 * 2^-8 * scale * sum |q_d k_d|, which is proportional to the keys' size, and p
with it.  The keys here are up to several times larger (their scales are what is
tested), so the class is multiplied by their root mean square where that is
above 1."""
import math
from dataclasses import replace

import numpy as np
import pytest
import torch

import _gpu
import block_sparse_paged_csr_gb300 as sa
import inputs
import oracle

pytestmark = pytest.mark.gpu

TORCH = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
HALF_BF16 = 2.0 ** -8


def scaled_workload(w, kind, act="f32", scales="pow2", seed=0, dirty=True):
    """Device tensors of workload `w` with K/V in 8 bits, and the f32 values
    they stand for.  Rows that no sequence reaches hold NaN codes (e4m3) or
    large ones."""
    rng = np.random.default_rng(seed + 77)
    t = _gpu.device_workload(replace(w, kv_dtype="f32"))
    t["q"] = t["q"].to(torch.bfloat16) if act == "bf16" else t["q"]
    live = np.zeros((w.num_pages, w.page_size), bool)
    for b in range(w.batch):
        n = int(w.used_kv_lens[b]) if w.pass_used else w.msb * w.block_size
        for p in range(min(-(-n // w.page_size), w.max_pages)):
            page = w.block_tables[b, p]
            if 0 <= page < w.num_pages:
                live[page, :max(0, min(n - p * w.page_size, w.page_size))] = True
    vals = {}
    for name in ("k", "v"):
        x = t[name].view(w.num_pages, w.hkv, w.page_size, w.head_dim)
        shape = (w.num_pages, w.hkv)
        if scales == "pow2":
            s = 2.0 ** rng.integers(-6, -3, shape)
        elif scales == "any":
            s = rng.uniform(0.02, 0.1, shape)
        elif scales == "wide":                   # of V: those of K set the scores' size
            s = 2.0 ** (rng.integers(-16, 5, shape) if name == "v" else rng.integers(-6, -3, shape))
        else:                                    # some pages stand for zeros
            s = np.where(rng.random(shape) < 0.3, 0.0, 0.04)
        s = torch.from_numpy(s.astype(np.float32)).cuda()
        gain = 30.0 if kind == "int8" else 90.0
        codes = (x * gain).round() if kind == "int8" else x * gain
        codes = codes.clamp(-127, 127).to(TORCH[kind])
        v = (codes.float() * s[:, :, None, None]).cpu().numpy()
        if dirty:
            dead = torch.from_numpy(~live).cuda()[:, None, :, None].expand_as(codes)
            raw = codes.view(torch.uint8)
            raw[dead] = 0x7F
        t[name], t[name + "s"] = codes, s
        v[~np.broadcast_to(live[:, None, :, None], v.shape)] = 0.0
        vals[name] = v
    return t, vals


def reference(w, t, vals):
    return oracle.attention(t["q"].float().cpu().numpy(), vals["k"], vals["v"], w.selected,
                            w.block_tables, w.cu_seqlens_q, w.used, w.hq, w.head_dim, w.block_size,
                            w.page_size, w.softmax_scale, w.causal)


def attend(w, t, **kw):
    out, lse, idx, parts = sa.sa_attention(
        t["q"], t["k"], t["v"], t["selected"], w.cu_seqlens_q, t["cu"], t["used"], t["bt"], w.hq,
        w.hkv, w.head_dim, w.block_size, w.page_size, w.softmax_scale, w.causal,
        k_scales=t["ks"], v_scales=t["vs"], **kw)
    assert sa.sa_get_status(idx) == 0
    assert out.dtype == t["q"].dtype and lse.dtype == torch.float32
    return out, lse, idx, parts


def kernel(w, kind):
    return sa.sa_attention_kernel_name(w.cu_seqlens_q, w.num_pages, w.hkv, w.hq, w.head_dim,
                                       w.block_size, w.page_size, kind, causal=w.causal)


def tc_tol(vals):
    k = vals["k"][vals["k"] != 0]
    return _gpu.TOL_TC * max(1.0, float(np.sqrt(np.mean(k.astype(np.float64) ** 2))))


def check(w, t, vals, tol, name="", **kw):
    out, lse, idx, parts = attend(w, t, **kw)
    ref, ref_lse, _, _ = reference(w, t, vals)
    got = out.float().cpu().numpy()
    assert np.isfinite(got).all()
    if t["q"].dtype == torch.bfloat16:
        tol += HALF_BF16
    _gpu.report(f"8-bit {name}", "out", got, ref)
    assert _gpu.row_error(got, ref) <= tol
    _gpu.compare_lse(lse.cpu().numpy(), ref_lse, min(tol, 1e-4) if tol < 1e-2 else tol)
    return out, lse


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("name", ["gqa_decode", "long_decode"])
def test_fused_decode(kind, act, name):
    w = inputs.small(name, seed=31)
    assert kernel(w, kind) == "fused_dec_kernel"
    t, vals = scaled_workload(w, kind, act)
    check(w, t, vals, _gpu.TOL_F32, f"{name} {kind} {act}")


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv,ps,bs,topk", [
    (1, 1, 16, 64, 3), (6, 2, 16, 16, 5), (8, 1, 32, 32, 4), (15, 3, 16, 128, 3),
    (32, 2, 64, 64, 6), (12, 1, 16, 64, 7), (18, 2, 128, 128, 2), (16, 1, 16, 32, 9),
    (4, 4, 256, 256, 2), (8, 8, 16, 64, 80)])
def test_fused_decode_geometries(kind, hq, hkv, ps, bs, topk):
    """Group sizes 1 to 16, pages of 16 to 256 keys, blocks of a page and of
    several, more ranks than a piece holds."""
    w = inputs.gqa_decode(41, batch=5, kv_min=max(bs * topk, 300), kv_max=max(bs * topk, 300) + 777,
                          hq=hq, hkv=hkv, page_size=ps, block_size=bs, topk=topk)
    assert kernel(w, kind) == "fused_dec_kernel"
    t, vals = scaled_workload(w, kind)
    check(w, t, vals, _gpu.TOL_F32, f"fused {hq}/{hkv} {ps}/{bs} {kind}")


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("scales", ["any", "wide", "zeros"])
@pytest.mark.parametrize("hq", [8, 24])
def test_fused_decode_scales(kind, scales, hq):
    w = inputs.gqa_decode(43, batch=4, kv_min=700, kv_max=1500, hq=hq, hkv=2, topk=8)
    t, vals = scaled_workload(w, kind, scales=scales)
    check(w, t, vals, _gpu.TOL_F32, f"fused scales {scales} {kind}")


def spread_workload(kind, hq, e, where, seed):
    """A decode batch in which one page of each sequence takes nearly all of the
    softmax (`where` "light") or as much of the output as the others (`where`
    "even") while its V scale is 2^-e of theirs, or (`where` "heavy") has a share
    of 2^-e of the softmax and a V scale of 2^e."""
    hkv, d, ps, bs, topk = 2, 128, 16, 64, 6
    w = inputs.gqa_decode(seed, batch=4, kv_min=500, kv_max=900, hq=hq, hkv=hkv, topk=topk)
    rng = np.random.default_rng(seed)
    sel = np.sort(np.argsort(rng.random((w.tq, hkv, 7)), axis=2)[:, :, :topk].astype(np.int32), axis=2)
    w = replace(w, selected=sel)
    t = _gpu.device_workload(replace(w, kv_dtype="f32"))
    # every lane points along one direction of signs, the page's keys too
    sign = rng.choice([-1.0, 1.0], (w.tq, hkv, d))
    q = np.repeat(sign, hq // hkv, axis=1) * rng.uniform(0.9, 1.1, (w.tq, hq, 1))
    t["q"] = torch.from_numpy(q.astype(np.float32)).cuda()
    shape = (w.num_pages, hkv, ps, d)
    k = rng.choice([-1.0, 0.0, 1.0], shape)
    v = np.round(rng.standard_normal(shape) * 30).clip(-100, 100)
    ks = np.full(shape[:2], 0.02)
    vs = np.ones(shape[:2])
    nat = e * math.log(2.0)
    gain = {"light": nat + 20.0, "even": nat, "heavy": -nat}[where]
    for i in range(w.tq):                     # (sequence i holds query i)
        for h in range(hkv):
            block = int(sel[i, h, rng.integers(topk)])
            page = w.block_tables[i, block * (bs // ps) + int(rng.integers(bs // ps))]
            c = 100.0
            k[page, h] = sign[i, h] * c
            # score gain = softmax_scale * d * c * ks
            ks[page, h] = gain / (w.softmax_scale * d * c)
            vs[page, h] = 2.0 ** (e if where == "heavy" else -e)
    vals = {}
    for name, x, s in (("k", k, ks), ("v", v, vs)):
        codes = torch.from_numpy(x).cuda().to(torch.float32).to(TORCH[kind])
        s = torch.from_numpy(s.astype(np.float32)).cuda()
        t[name], t[name + "s"] = codes, s
        vals[name] = (codes.double() * s.double()[:, :, None, None] if kind == "int8" else
                      codes.float().double() * s.double()[:, :, None, None]).float().cpu().numpy()
    return w, t, vals


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hq", [8, 24])
@pytest.mark.parametrize("where", ["light", "even", "heavy"])
@pytest.mark.parametrize("e", [4, 12, 20, 28, 40, 60])
def test_fused_decode_scales_far_apart(kind, hq, where, e):
    """V scales up to 2^60 apart in one piece, the output from either end: what
    a page adds keeps f32's class whatever the other pages' scales are, and
    however the ranks are cut."""
    w, t, vals = spread_workload(kind, hq, e, where, 71)
    assert kernel(w, kind) == "fused_dec_kernel"
    ref, ref_lse, _, _ = reference(w, t, vals)
    size = np.abs(ref).max(axis=-1, keepdims=True)        # (no floor: outputs may be small)
    for split in (0, 1, 4, 64):
        out, lse, _, _ = attend(w, t, split_edges=split)
        got = out.cpu().numpy().astype(np.float64)
        assert (np.abs(got - ref) / size).max() <= _gpu.TOL_F32
        _gpu.compare_lse(lse.cpu().numpy(), ref_lse, 1e-4)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hq", [8, 24])
@pytest.mark.parametrize("v_scale", [0.0, 2.0 ** -126, -(2.0 ** -60), 2.0 ** 100])
def test_fused_decode_scales_at_the_ends(kind, hq, v_scale):
    """V scales at the ends of f32's range, negative, and 0 for half of the pages
    (their keys count in the softmax all the same)."""
    w = inputs.gqa_decode(73, batch=3, kv_min=400, kv_max=700, hq=hq, hkv=2, topk=5)
    t, vals = scaled_workload(w, kind, dirty=False)
    s = torch.full_like(t["vs"], v_scale)
    if v_scale == 0.0:
        s[::2] = 0.5
    vals["v"] = (t["v"].float() * s[:, :, None, None]).cpu().numpy()
    t["vs"] = s
    ref, ref_lse, _, _ = reference(w, t, vals)
    size = np.abs(ref).max(axis=-1, keepdims=True)
    for split in (0, 1, 64):
        out, lse, _, _ = attend(w, t, split_edges=split)
        got = out.cpu().numpy().astype(np.float64)
        # (outputs near 2^-126 are held in steps of 2^-149)
        assert (np.abs(got - ref) <= _gpu.TOL_F32 * size + 2.0 ** -148).all()
        _gpu.compare_lse(lse.cpu().numpy(), ref_lse, 1e-4)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hq", [8, 24])
@pytest.mark.parametrize("page_size", [16, 64])
def test_fused_decode_scale_beyond_reach(kind, hq, page_size):
    """A page whose V scale is 2^160 times the others' and whose keys have 2^-250
    of the softmax adds nothing, and no NaN (0 times infinity) either, whether
    it comes first, where the sequence ends inside it, or last."""
    w = inputs.gqa_decode(77, batch=3, kv_min=400, kv_max=700, hq=hq, hkv=2, topk=5,
                          page_size=page_size)
    t, vals = scaled_workload(w, kind, dirty=False)
    shape = (w.num_pages, 2, page_size, 128)
    sign = np.random.default_rng(7).choice([-1.0, 1.0], 128)
    t["q"] = torch.from_numpy(np.tile(sign, (w.tq, hq, 1)).astype(np.float32)).cuda()
    k = np.random.default_rng(8).choice([-1.0, 0.0, 1.0], shape)
    ks, vs = np.full(shape[:2], 0.02), np.full(shape[:2], 2.0 ** -60)
    for b in range(3):
        for h in range(2):                   # head 0: the first rank's last page; head 1: the last rank's
            last = (int(w.used_kv_lens[b]) - 1) // page_size
            page = w.block_tables[b, last if h == 0 else w.selected[b, h, -1] * (64 // page_size)]
            k[page, h] = sign * 100.0
            ks[page, h] = -250 * math.log(2.0) / (w.softmax_scale * 128 * 100.0)
            vs[page, h] = 2.0 ** 100
    for name, x, s in (("k", torch.from_numpy(k).float(), ks), ("v", t["v"].float().cpu(), vs)):
        codes = x.cuda().to(TORCH[kind])
        t[name], t[name + "s"] = codes, torch.from_numpy(s.astype(np.float32)).cuda()
        vals[name] = (codes.float() * t[name + "s"][:, :, None, None]).cpu().numpy()
    ref, ref_lse, _, _ = reference(w, t, vals)
    size = np.abs(ref).max(axis=-1, keepdims=True)
    for split in (0, 1, 64):                 # (64: one piece of all ranks)
        out, lse, _, _ = attend(w, t, split_edges=split)
        got = out.cpu().numpy().astype(np.float64)
        assert (np.abs(got - ref) <= _gpu.TOL_F32 * size).all()
        _gpu.compare_lse(lse.cpu().numpy(), ref_lse, 1e-4)


@pytest.mark.parametrize("split", [1, 3, 64])
@pytest.mark.parametrize("partial", [None, "bf16"])
def test_fused_decode_pieces(split, partial):
    w = inputs.small("long_decode", seed=33)
    t, vals = scaled_workload(w, "e4m3", "bf16")
    check(w, t, vals, _gpu.TOL_F32 if partial is None else HALF_BF16, f"pieces {split} {partial}",
          split_edges=split, partial_dtype=partial)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("act,qscale", [("f32", 1e-20), ("f32", 100.0), ("bf16", 1e-6), ("f32", 0.0)])
def test_fused_decode_query_range(kind, act, qscale):
    """Queries far from 1 (split into f16 parts after a power of two)."""
    w = inputs.small("gqa_decode", seed=35)
    w = replace(w, softmax_scale=w.softmax_scale / (qscale if qscale > 0 else 1.0))
    t, vals = scaled_workload(w, kind)
    t["q"] = (t["q"] * qscale).to(torch.bfloat16 if act == "bf16" else torch.float32)
    check(w, t, vals, _gpu.TOL_F32, f"q x {qscale} {kind}")


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_empty_rows_and_missing_pages(kind):
    """A sequence of length 0, one of a single key, one whose ranks are all
    empty, missing pages inside a block, and queries of fewer sequences than
    the batch."""
    w = inputs.gqa_decode(45, batch=6, kv_min=300, kv_max=900, hq=8, hkv=2, topk=5)
    lens = w.used_kv_lens.copy()
    lens[0], lens[1] = 0, 1
    sel = w.selected.copy()
    sel[1] = -1
    sel[1, :, 2] = 0
    sel[2] = -1
    bt = w.block_tables.copy()
    bt[3, ::3] = -1
    bt[4, :] = -1
    qo = w.qo_lens.copy()
    qo[5] = 0
    w = replace(w, used_kv_lens=lens, selected=sel[:5].copy(), block_tables=bt, qo_lens=qo)
    t, vals = scaled_workload(w, kind)
    out, lse = check(w, t, vals, _gpu.TOL_F32, f"empty {kind}")
    for i in (0, 2, 4):
        assert (out[i] == 0).all() and (lse[i] == -math.inf).all()


GENERAL = [  # batch, qo, kv, hq, hkv, d, ps, bs, topk
    (2, 3, 200, 6, 2, 64, 16, 32, 4), (1, 1, 90, 4, 4, 32, 4, 16, 6), (2, 2, 130, 5, 1, 48, 8, 48, 2),
    (1, 5, 300, 2, 1, 256, 16, 64, 3), (3, 1, 70, 3, 3, 16, 2, 8, 5), (2, 2, 500, 8, 2, 128, 16, 64, 5)]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("batch,qo,kv,hq,hkv,d,ps,bs,topk", GENERAL)
def test_general_kernel(kind, act, batch, qo, kv, hq, hkv, d, ps, bs, topk):
    w = inputs.chunked_prefill(51, batch=batch, qo_len=qo, kv_len=kv, hq=hq, hkv=hkv, head_dim=d,
                               page_size=ps, block_size=bs, topk=topk)
    t, vals = scaled_workload(w, kind, act, scales="any")
    check(w, t, vals, _gpu.TOL_F32, f"general {d} {ps}/{bs} {kind} {act}",
          path=sa.PATH_CUDA_CORE)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("name", ["chunked_prefill", "skewed"])
def test_tensor_cores(kind, act, name):
    w = inputs.small(name, seed=53)
    assert kernel(w, kind) == "forward_tc_kernel"
    t, vals = scaled_workload(w, kind, act)
    check(w, t, vals, tc_tol(vals), f"{name} {kind} {act}")
    check(w, t, vals, tc_tol(vals), f"{name} {kind} {act} bf16 partials", partial_dtype="bf16")


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_tensor_cores_odd_lengths(kind):
    """Lengths that end inside pages, rows of padding, scales of any value."""
    w = inputs.skewed(55, batch=3, qo_len=37, kv_len=1999, hq=16, hkv=2, topk=6)
    w = replace(w, used_kv_lens=np.array([1999, 1003, 64], np.int32))
    t, vals = scaled_workload(w, kind, "bf16", scales="any")
    check(w, t, vals, tc_tol(vals), f"odd {kind}")


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("scales", ["pow2", "any", "signs"])
@pytest.mark.parametrize("bs,qo,lens", [(64, 37, (1999, 1003, 64)), (128, 300, (1999, 300, 777))])
def test_tensor_cores_scales_lose_nothing(kind, scales, bs, qo, lens):
    """With bf16 queries, whatever the scales, what the tensor-core kernel rounds
    is P and the output, half a step of bf16 (2^-8) each: an element is off by at
    most 2^-8 sum p |v| / sum p + 2^-8 |out|, besides the sums' f32 class."""
    make = inputs.skewed if bs == 64 else inputs.chunked_prefill
    w = make(75, batch=3, qo_len=qo, kv_len=1999, hq=16, hkv=2, topk=6, block_size=bs)
    w = replace(w, used_kv_lens=np.array(lens, np.int32))
    assert kernel(w, kind) == "forward_tc_kernel"
    t, vals = scaled_workload(w, kind, "bf16", scales="any" if scales == "signs" else scales)
    if scales == "signs":
        for name in ("ks", "vs"):
            sign = torch.from_numpy(np.random.default_rng(len(name)).choice([-1.0, 1.0], t[name].shape))
            t[name] = t[name] * sign.float().cuda()
            vals[name[0]] = vals[name[0]] * sign.numpy()[:, :, None, None].astype(np.float32)
    out, lse, _, _ = attend(w, t)
    ref, ref_lse, _, _ = reference(w, t, vals)
    size, _, _, _ = reference(w, t, dict(k=vals["k"], v=np.abs(vals["v"])))
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - ref)
    assert (err <= (HALF_BF16 + _gpu.TOL_F32) * size + HALF_BF16 * np.abs(ref)).all()
    _gpu.compare_lse(lse.cpu().numpy(), ref_lse, _gpu.TOL_F32)


@pytest.mark.parametrize("path", [sa.PATH_AUTO, sa.PATH_CUDA_CORE])
def test_steps_one_by_one(path):
    """sa_forward and sa_combine, and sa_forward_combine, on a built index."""
    w = inputs.small("chunked_prefill", seed=57)
    t, vals = scaled_workload(w, "int8", "f32")
    ref, ref_lse, _, _ = reference(w, t, vals)
    tol = tc_tol(vals) if path == sa.PATH_AUTO else _gpu.TOL_F32
    idx = sa.sa_build_index(t["selected"], w.cu_seqlens_q, t["cu"], t["used"], w.max_pages,
                            w.block_size, w.page_size)
    kw = dict(k_scales=t["ks"], v_scales=t["vs"], path=path)
    o, m, l = sa.sa_forward(t["q"], t["k"], t["v"], idx, t["bt"], t["cu"], t["used"], w.hq, w.hkv,
                            w.head_dim, w.block_size, w.page_size, w.softmax_scale, w.causal, **kw)
    out, lse = sa.sa_combine(idx, o, m, l, w.hq, w.head_dim)
    assert _gpu.row_error(out.cpu().numpy(), ref) <= tol
    out2, lse2, _ = sa.sa_forward_combine(
        t["q"], t["k"], t["v"], idx, t["selected"], w.cu_seqlens_q, t["cu"], t["used"], t["bt"],
        w.hq, w.head_dim, w.block_size, w.page_size, w.softmax_scale, w.causal, **kw)
    assert sa.sa_get_status(idx) == 0
    assert _gpu.row_error(out2.cpu().numpy(), ref) <= tol
    _gpu.compare_lse(lse2.cpu().numpy(), ref_lse, tol)


def test_arguments():
    w = inputs.small("gqa_decode", seed=59)
    t, _ = scaled_workload(w, "int8")
    with pytest.raises(ValueError):
        attend(w, dict(t, ks=None))
    with pytest.raises(ValueError):
        attend(w, dict(t, vs=t["vs"][:-1].contiguous()))
    with pytest.raises(TypeError):
        attend(w, dict(t, ks=t["ks"].double()))
    with pytest.raises(TypeError):
        attend(w, dict(t, q=t["q"].half()))
    with pytest.raises(TypeError):
        attend(w, t, out=torch.empty_like(t["q"], dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        attend(w, dict(t, v=t["v"].float()))
    f = _gpu.device_workload(w)
    with pytest.raises(ValueError):
        attend(w, dict(f, ks=t["ks"], vs=t["vs"]))
    with pytest.raises(sa.SAError):      # one query per sequence only
        w2 = inputs.small("chunked_prefill", seed=59)
        t2, _ = scaled_workload(w2, "int8")
        attend(w2, t2, path=sa.PATH_FUSED_DECODE)


@pytest.mark.parametrize("name", ["gqa_decode", "chunked_prefill"])
def test_graph_and_streams(name):
    """A captured step replayed on new contents, and a call on a stream of the
    caller's, give what an eager call gives, bit for bit."""
    w = inputs.small(name, seed=61)
    t, _ = scaled_workload(w, "e4m3", "bf16")
    args = (t["q"], t["k"], t["v"], t["selected"], w.cu_seqlens_q, t["cu"], t["used"], t["bt"], w.hq,
            w.hkv, w.head_dim, w.block_size, w.page_size, w.softmax_scale, w.causal)
    g = sa.AttentionGraph(*args, k_scales=t["ks"], v_scales=t["vs"])
    for seed in range(2):
        t["q"].copy_(torch.randn(t["q"].shape, device="cuda"))
        t["ks"].mul_(2.0)
        ref, ref_lse, _, _ = attend(w, t)
        out, lse = g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out, lse, _, _ = attend(w, t)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_serving_steps(kind, act):
    """The operators in the order a server calls them: a prompt is stored,
    its blocks' bounds taken, each query's blocks selected and attended to,
    then single tokens, step by step.  Every step's output against the oracle
    on the cache's values and the selection that was made."""
    batch, hkv, g, d, ps, bs, topk = 3, 2, 4, 128, 16, 64, 5
    hq = hkv * g
    gen = torch.Generator(device="cuda").manual_seed(3)
    prompt = np.array([200, 513, 64])
    steps = 4
    cols = -(-int(prompt.max() + steps) // bs)
    max_pages = cols * (bs // ps)
    perm = np.random.default_rng(4).permutation(batch * max_pages).astype(np.int32)
    bt = torch.from_numpy(perm.reshape(batch, max_pages)).cuda()
    rows = torch.arange(batch * cols, dtype=torch.int32, device="cuda").view(batch, cols)
    shape = (batch * max_pages, hkv, ps, d)
    kp = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(TORCH[kind])
    vp = kp.clone()
    ks, vs = torch.zeros(shape[:2], device="cuda"), torch.zeros(shape[:2], device="cuda")
    bounds = torch.zeros((batch * cols, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    lens = prompt.copy()
    qo = prompt.copy()
    for step in range(steps):
        cu = np.concatenate([[0], np.cumsum(qo)]).astype(np.int64)
        tq = int(cu[-1])
        cud = torch.from_numpy(cu).cuda()
        used = torch.from_numpy(lens.astype(np.int32)).cuda()
        qkv = torch.randn((tq, hq + 2 * hkv, d), generator=gen, device="cuda")
        qkv = qkv.to(torch.bfloat16 if act == "bf16" else torch.float32)
        q = qkv[:, :hq].contiguous()
        sa.sa_store_kv(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kp, vp, bt, cu, cud, used,
                       k_scales=ks, v_scales=vs, status=status)
        sa.sa_block_bounds(kp, bt, cu, cud, used, bounds, rows, bs, k_scales=ks, status=status)
        sel = sa.sa_select_blocks(q, bounds, rows, cu, cud, used, bs, topk, True, sink_blocks=1,
                                  local_blocks=1, status=status)
        out, lse, idx, _ = sa.sa_attention(q, kp, vp, sel, cu, cud, used, bt, hq, hkv, d, bs, ps,
                                           1 / math.sqrt(d), True, k_scales=ks, v_scales=vs)
        assert sa.sa_get_status(idx) == 0 and int(status) == 0
        selected = sel.cpu().numpy()
        for b in range(batch):
            pos = np.arange(lens[b] - qo[b], lens[b])
            own = pos // bs
            s = selected[cu[b]:cu[b + 1]]
            assert (s[:, :, 0] == 0).all()
            assert (s.max(2) == own[:, None]).all()
            assert (((s >= 0).sum(2)) == np.minimum(own + 1, topk)[:, None]).all()
        kf = np.nan_to_num((kp.float() * ks[:, :, None, None]).cpu().numpy())
        vf = np.nan_to_num((vp.float() * vs[:, :, None, None]).cpu().numpy())
        ref, ref_lse, _, _ = oracle.attention(q.float().cpu().numpy(), kf, vf, selected,
                                              bt.cpu().numpy(), cu, used.cpu().numpy(), hq, d, bs,
                                              ps, 1 / math.sqrt(d), True)
        tol = (_gpu.TOL_TC if step == 0 else _gpu.TOL_F32) + (HALF_BF16 if act == "bf16" else 0.0)
        assert _gpu.row_error(out.float().cpu().numpy(), ref) <= tol
        lens = lens + 1
        qo = np.ones(batch, np.int64)


def test_every_launch_names_its_device(monkeypatch):
    """Each call to the library that launches or synchronises is made with the
    device of its tensors as the current one."""
    w = inputs.small("gqa_decode", seed=63)
    made = set()
    on = sa._on

    def record(dev, fn, *args):
        assert dev == torch.device("cuda", 0)
        made.add(fn.__name__)
        return on(dev, fn, *args)

    monkeypatch.setattr(sa, "_on", record)
    wide = _gpu.device_workload(w)
    eight, _ = scaled_workload(w, "int8")
    for t, kw in ((wide, {}), (eight, dict(k_scales=eight["ks"], v_scales=eight["vs"]))):
        for partial in (None, "bf16"):
            args = (w.hq, w.hkv, w.head_dim, w.block_size, w.page_size, w.softmax_scale, w.causal)
            idx = sa.sa_build_index(t["selected"], w.cu_seqlens_q, t["cu"], t["used"], w.max_pages,
                                    w.block_size, w.page_size)
            sa.sa_build_index_no_alloc(t["selected"], w.cu_seqlens_q, t["cu"], t["used"], idx,
                                       w.max_pages, w.block_size, w.page_size)
            o, m, l = sa.sa_forward(t["q"], t["k"], t["v"], idx, t["bt"], t["cu"], t["used"], *args,
                                    partial_dtype=partial, **kw)
            sa.sa_combine(idx, o, m, l, w.hq, w.head_dim)
            sa.sa_forward_combine(t["q"], t["k"], t["v"], idx, t["selected"], w.cu_seqlens_q, t["cu"],
                                  t["used"], t["bt"], args[0], *args[2:], partial_dtype=partial, **kw)
            sa.sa_attention(t["q"], t["k"], t["v"], t["selected"], w.cu_seqlens_q, t["cu"], t["used"],
                            t["bt"], *args, partial_dtype=partial, **kw)
            assert sa.sa_get_status(idx) == 0
            sa.sa_clear_status(idx)
    assert made == {"sa_build_index", "sa_build_index_no_alloc", "sa_forward", "sa_forward_ex",
                    "sa_forward_scaled", "sa_combine", "sa_combine_ex", "sa_forward_combine",
                    "sa_forward_combine_ex", "sa_forward_combine_scaled", "sa_attention",
                    "sa_attention_ex", "sa_attention_scaled", "sa_get_status", "sa_clear_status"}


@pytest.mark.parametrize("current,device,switched", [(0, 0, False), (1, 0, True), (0, 1, True)])
def test_device_switch(monkeypatch, current, device, switched):
    """_on makes the tensors' device current where it is not (the devices are
    names here: the call is a Python function)."""
    seen = []

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            seen.append(("in", self.d.index))

        def __exit__(self, *a):
            seen.append(("out", self.d.index))

    monkeypatch.setattr(sa, "_current_device", lambda: current)
    monkeypatch.setattr(sa.torch.cuda, "device", Device)
    assert sa._on(torch.device("cuda", device), lambda x: x + 1, 4) == 5
    assert seen == ([("in", device), ("out", device)] if switched else [])


def test_buffers_belong_to_the_stream_of_the_call():
    """What a call allocates comes from the stream that it names, where memory
    that the current stream freed and still uses is not handed out."""
    w = inputs.small("gqa_decode", seed=65)
    t, vals = scaled_workload(w, "int8")
    ref, ref_lse, _, _ = reference(w, t, vals)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, lse, idx, parts = attend(w, t, stream=side)
    bounds = torch.zeros((4, w.hkv, 2, w.head_dim), dtype=torch.bfloat16, device="cuda")
    tables = torch.zeros((w.batch, 4), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    sel = sa.sa_select_blocks(t["q"], bounds, tables, w.cu_seqlens_q, t["cu"], t["used"],
                              w.block_size, 2, True, stream=side)
    i2 = sa.sa_build_index(t["selected"], w.cu_seqlens_q, t["cu"], t["used"], w.max_pages,
                           w.block_size, w.page_size, stream=side)
    o, m, l = sa.sa_forward(t["q"], t["k"], t["v"], i2, t["bt"], t["cu"], t["used"], w.hq, w.hkv,
                            w.head_dim, w.block_size, w.page_size, w.softmax_scale, w.causal,
                            k_scales=t["ks"], v_scales=t["vs"], stream=side)
    out2, lse2 = sa.sa_combine(i2, o, m, l, w.hq, w.head_dim, stream=side)
    out3, lse3, p3 = sa.sa_forward_combine(
        t["q"], t["k"], t["v"], i2, t["selected"], w.cu_seqlens_q, t["cu"], t["used"], t["bt"], w.hq,
        w.head_dim, w.block_size, w.page_size, w.softmax_scale, w.causal, k_scales=t["ks"],
        v_scales=t["vs"], stream=side)
    side.synchronize()
    for x in (out, out2, out3):
        assert _gpu.row_error(x.cpu().numpy(), ref) <= _gpu.TOL_F32
    segments = torch.cuda.memory_snapshot()
    for x in (out, lse, *parts, idx.totals, idx.workspace, idx.edges, sel, i2.inv, o, m, l, out2, lse2,
              out3, lse3, *p3):
        of = [s["stream"] for s in segments
              if s["address"] <= x.data_ptr() < s["address"] + s["total_size"]]
        assert of == [side.cuda_stream]


@pytest.mark.parametrize("kind", ["f32", "int8"])
def test_tensors_smaller_than_the_call(kind):
    """Tables, lengths, queries and buffers that are too small, of another layout
    or type are refused before any launch."""
    w = inputs.small("gqa_decode", seed=67)
    if kind == "f32":
        t = _gpu.device_workload(w)
        kw = {}
    else:
        t, _ = scaled_workload(w, kind)
        kw = dict(k_scales=t["ks"], v_scales=t["vs"])
    sizes = (w.hq, w.hkv, w.head_dim, w.block_size, w.page_size, w.softmax_scale, w.causal)

    def attention(t, **more):
        return sa.sa_attention(t["q"], t["k"], t["v"], t["selected"], w.cu_seqlens_q, t["cu"],
                               t["used"], t["bt"], *sizes, **kw, **more)

    def steps(t, **more):
        return sa.sa_forward_combine(t["q"], t["k"], t["v"], idx, t["selected"], w.cu_seqlens_q,
                                     t["cu"], t["used"], t["bt"], w.hq, *sizes[2:], **kw, **more)

    def forward(t, **more):
        return sa.sa_forward(t["q"], t["k"], t["v"], idx, t["bt"], t["cu"], t["used"], *sizes, **kw,
                             **more)

    out, lse, idx, parts = attention(t)
    bad = dict(q=t["q"][:-1], cu=t["cu"][:-1], used=t["used"][:-1], bt=t["bt"].t().contiguous().t())
    short = dict(bt=t["bt"][:-1], selected=t["selected"][:-1])
    for call in (attention, steps, forward):
        for name, x in {**bad, "bt": short["bt"]}.items():
            if call is attention and name == "bt":
                continue
            with pytest.raises(ValueError):
                call({**t, name: x})
        with pytest.raises(ValueError):
            call({**t, "bt": bad["bt"]})
        with pytest.raises(TypeError):
            call({**t, "bt": t["bt"].long()})
        with pytest.raises(TypeError):
            call({**t, "cu": t["cu"].int()})
    for call in (attention, steps):
        with pytest.raises(ValueError):
            call({**t, "selected": t["selected"][:, :1].contiguous()})
        with pytest.raises(ValueError):
            call(t, out=out[:-1])
        with pytest.raises(ValueError):
            call(t, lse=lse[:-1])
        with pytest.raises(TypeError):
            call(t, lse=lse.double())
        for i in range(3):
            with pytest.raises(ValueError):
                call(t, partials=tuple(p[:-1] if i == x else p for x, p in enumerate(parts)))
    with pytest.raises(ValueError):
        attention({**t, "bt": short["bt"]})
    with pytest.raises(ValueError):
        forward(t, m_partial=parts[1][:-1])
    small = sa.allocate_index(w.tq, w.hkv, w.topk - 1, w.batch, w.max_pages, w.block_size, w.page_size,
                              "cuda")
    with pytest.raises(ValueError):
        attention(t, index=small)
    with pytest.raises(ValueError):
        sa.sa_build_index(t["selected"], w.cu_seqlens_q, t["cu"], t["used"], w.max_pages, w.block_size,
                          w.page_size, index=small)
    with pytest.raises(ValueError):
        sa.sa_combine(idx, *parts, w.hq, w.head_dim, out=out[:-1].float())
    torch.cuda.synchronize()


def test_stream_by_its_handle():
    """A stream that is not torch's own, known by its handle only."""
    import types

    w = inputs.small("gqa_decode", seed=69)
    t, vals = scaled_workload(w, "int8")
    ref, _, _, _ = reference(w, t, vals)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, _, idx, _ = attend(w, t, stream=types.SimpleNamespace(cuda_stream=side.cuda_stream))
    torch.cuda.synchronize()
    assert _gpu.row_error(out.cpu().numpy(), ref) <= _gpu.TOL_F32
