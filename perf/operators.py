"""What the measurements of the cache and block-selection operators run.

Four operators of a sparse-attention serving step, in the order a server calls
them: new tokens go into the paged cache (``store``), the bounds of the blocks
they touched are renewed (``bounds``), every query picks its blocks by those
bounds (``select``), and the attention runs over a cache held in 8 bits with a
scale for each page and kv head (``attend``).

``own`` False computes each operator in plain torch; True calls the library.
"""
import math

import numpy as np
import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
         "int8": torch.int8}


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token for each of 64 running sequences: the append of a decode step (latency)
        dict(name="store_decode", op="store", batch=64, qo_min=1, qo_max=1, kv_min=300,
             kv_max=2000, hq=32, hkv=8, d=128, ps=16, bs=64, cache="e4m3", act="bf16"),
        # a prompt chunk of four long sequences into pages of 64, f32 activations
        dict(name="store_prompt", op="store", batch=4, qo_min=1501, qo_max=2048, kv_min=4096,
             kv_max=8192, hq=64, hkv=8, d=128, ps=64, bs=128, cache="int8", act="f32"),
        # the block that each of 128 decoding sequences just wrote to
        dict(name="bounds_decode", op="bounds", batch=128, qo_min=1, qo_max=1, kv_min=500,
             kv_max=3000, hq=64, hkv=8, d=128, ps=16, bs=64, cache="e4m3", act="f32"),
        # every block of freshly stored prompts
        dict(name="bounds_prompt", op="bounds", batch=4, qo_min=20001, qo_max=32768, kv_min=20001,
             kv_max=32768, hq=64, hkv=8, d=128, ps=64, bs=128, cache="int8", act="f32"),
        # block selection of the grouped-query decode batch
        dict(name="select_decode", op="select", batch=64, qo_min=1, qo_max=1, kv_min=4096,
             kv_max=32768, hq=32, hkv=8, d=128, ps=16, bs=64, topk=16, act="f32"),
        # ... of the long-context decode batch
        dict(name="select_long", op="select", batch=128, qo_min=1, qo_max=1, kv_min=65536,
             kv_max=131072, hq=64, hkv=8, d=128, ps=16, bs=64, topk=64, act="bf16"),
        # ... of chunked prefill
        dict(name="select_prefill", op="select", batch=4, qo_min=2048, qo_max=2048, kv_min=32768,
             kv_max=32768, hq=64, hkv=8, d=128, ps=64, bs=128, topk=32, act="f32"),
        # attention of a few sequences with a small head and an odd group: latency
        dict(name="attend_small", op="attend", batch=3, qo_min=1, qo_max=1, kv_min=90, kv_max=700,
             hq=6, hkv=2, d=64, ps=16, bs=32, topk=4, cache="int8", act="f32"),
        # the grouped-query decode batch
        dict(name="attend_decode", op="attend", batch=64, qo_min=1, qo_max=1, kv_min=4096,
             kv_max=32768, hq=32, hkv=8, d=128, ps=16, bs=64, topk=16, cache="e4m3", act="f32"),
        # long-context decode, both 8-bit types
        dict(name="attend_long", op="attend", batch=128, qo_min=1, qo_max=1, kv_min=65536,
             kv_max=131072, hq=64, hkv=8, d=128, ps=16, bs=64, topk=64, cache="e4m3", act="bf16"),
        dict(name="attend_long_int8", op="attend", batch=96, qo_min=1, qo_max=1, kv_min=20000,
             kv_max=50000, hq=64, hkv=8, d=128, ps=16, bs=64, topk=64, cache="int8", act="f32"),
        # a prompt chunk over its own selection
        dict(name="attend_prefill", op="attend", batch=2, qo_min=700, qo_max=1024, kv_min=16384,
             kv_max=32768, hq=64, hkv=8, d=128, ps=64, bs=128, topk=32, cache="e4m3", act="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "bounds", "select", "attend"])
    decode = rng.random() < 0.6
    hkv = rng.choice([1, 2, 4, 8])
    bs, ps = rng.choice([(64, 16), (64, 32), (64, 64), (128, 16), (128, 64), (32, 16)])
    d = rng.choice([128, 128, 128, 64])
    batch = _log(rng, 1, 100) if decode else rng.randint(1, 4)
    qo = 1 if decode else _log(rng, 2, 500 if op == "attend" else 2000)
    top = 30000 if op != "store" else 8000
    kv = [_log(rng, 50, top) for _ in range(2)]
    c = dict(op=op, batch=batch, qo_min=1 if decode else max(1, qo // 2), qo_max=qo,
             kv_min=max(min(kv), qo), kv_max=max(max(kv), qo),
             hq=hkv * rng.choice([1, 2, 3, 4, 5, 8] if d == 64 or decode else [1, 2, 4, 8]),
             hkv=hkv, d=d, ps=ps, bs=bs, act=rng.choice(["f32", "bf16"]))
    if op in ("select", "attend"):
        c["topk"] = _log(rng, 2, 40)
    if op != "select":
        c["cache"] = rng.choice(["e4m3", "int8"])
    if op == "attend" and not decode:
        c["act"] = "bf16"        # prompts run in bf16 activations on the tensor cores
    return c


# ----------------------------------------------------------------------------- inputs

def _lengths(case, seed):
    """New tokens and length of every sequence: of the case's own making, in the
    seed's order, so that the outputs of every seed have the same shapes."""
    rng = np.random.default_rng(case["batch"] + case["kv_max"])
    qo = rng.integers(case["qo_min"], case["qo_max"] + 1, case["batch"])
    lk = np.maximum(rng.integers(case["kv_min"], case["kv_max"] + 1, case["batch"]), qo)
    order = np.random.default_rng(seed).permutation(len(qo))
    return qo[order].astype(np.int64), lk[order].astype(np.int32)


def _tables(lk, per, gen):
    """[batch, columns] table of a randomly permuted pool with just the entries
    the lengths need (-1 behind them), and the pool's size."""
    live = torch.from_numpy(-(-lk.astype(np.int64) // per))
    cols = int(live.max())
    there = torch.arange(cols)[None, :] < live[:, None]
    n = int(live.sum())
    t = torch.full((len(lk), cols), -1, dtype=torch.int32, device="cuda")
    t[there.cuda()] = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
    return t, n


def _codes(shape, kind, gen):
    """Normal values in 8 bits, made 2^28 elements at a time."""
    out = torch.empty(shape, dtype=TORCH[kind], device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for at in range(0, flat.numel(), step):
        x = torch.randn(min(step, flat.numel() - at), generator=gen, device="cuda")
        flat[at:at + step] = (x.mul_(28.0).round_().clamp_(-127, 127) if kind == "int8"
                              else x.mul_(96.0).clamp_(-448, 448)).to(TORCH[kind])
    return out


def _scales(shape, kind, gen):
    e = torch.randint(-6, -3, shape, generator=gen, device="cuda")
    return torch.exp2((e if kind == "int8" else e - 2).float())


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = case
    qo, lk = _lengths(c, seed)
    cu = np.concatenate([[0], np.cumsum(qo)]).astype(np.int64)
    tq, hq, hkv, d, ps, bs = int(cu[-1]), c["hq"], c["hkv"], c["d"], c["ps"], c["bs"]
    s = dict(case=c, cu_host=cu, cu=torch.from_numpy(cu).cuda(), used=torch.from_numpy(lk).cuda(),
             kept={})
    act = TORCH[c["act"]]
    per = bs // ps
    if c["op"] != "select":
        # whole blocks of pages, so that the table's rows hold whole blocks
        s["bt"], n = _tables(-(-lk // bs) * bs, ps, gen)
        live = torch.arange(s["bt"].shape[1], device="cuda")[None, :] * ps < s["used"][:, None]
        s["bt"] = torch.where(live, s["bt"], -1)
        shape = (n, hkv, ps, d)
    if c["op"] == "store":
        # rows as a fused projection leaves them: K and V are slices of one tensor; keys have
        # channels of unlike size
        qkv = torch.randn((tq, hq + 2 * hkv, d), generator=gen, device="cuda")
        qkv *= torch.exp(0.5 * torch.randn((hq + 2 * hkv, d), generator=gen, device="cuda"))
        qkv = qkv.to(act)
        s["k"], s["v"] = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if c["op"] in ("store", "attend", "bounds"):
        s["kp"] = _codes(shape, c["cache"], gen)
        s["ks"] = _scales((n, hkv), c["cache"], gen)
    if c["op"] in ("store", "attend"):
        s["vp"] = _codes(shape, c["cache"], gen)
        s["vs"] = _scales((n, hkv), c["cache"], gen)
    if c["op"] in ("select", "bounds"):
        s["rows"], n = _tables(lk, bs, gen)
        if c["op"] == "bounds":
            s["bounds"] = torch.zeros((n, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
        else:
            # extremes of a block's keys around a centre of the block's own
            mid = torch.randn((n, hkv, 1, d), generator=gen, device="cuda")
            half = 1.5 + torch.rand((n, hkv, 1, d), generator=gen, device="cuda")
            s["bounds"] = torch.cat([mid - half, mid + half], 2).to(torch.bfloat16)
            del mid, half
    if c["op"] in ("select", "attend"):
        s["q"] = torch.randn((tq, hq, d), generator=gen, device="cuda").to(act)
    if c["op"] == "attend":
        # distinct blocks of those a query sees, its own (last) one among them, one rank in
        # ten left empty
        _, pos = _positions(s)
        nblk = pos // bs + 1
        x = torch.rand((tq, hkv, -(-int(lk.max()) // bs)), generator=gen, device="cuda")
        col = torch.arange(x.shape[2], device="cuda")
        x = torch.where(col < nblk[:, None, None], x, -1.0)
        x = torch.where(col == nblk[:, None, None] - 1, 2.0, x)
        v, i = x.topk(min(c["topk"], x.shape[2]), dim=2)
        empty = torch.rand(v.shape, generator=gen, device="cuda") < 0.1
        i = torch.where((v < 0) | ((v < 2) & empty), -1, i)
        s["selected"] = torch.full((tq, hkv, c["topk"]), -1, dtype=torch.int32, device="cuda")
        s["selected"][:, :, :i.shape[2]] = i.to(torch.int32)
    return s


def _positions(s):
    """Sequence and position in it of every query or new token."""
    cu, used = s["cu"], s["used"].long()
    i = torch.arange(int(s["cu_host"][-1]), device="cuda")
    b = torch.searchsorted(cu, i, right=True) - 1
    return b, used[b] - (cu[b + 1] - cu[b]) + i - cu[b]


# ----------------------------------------------------------------------------- plain forms

def _store_plain(s):
    """Per (page, head): the smallest power of two that holds the page's new
    rows, or the page's own where that is larger; codes to the nearest."""
    c = s["case"]
    hkv, d, ps, kind = c["hkv"], c["d"], c["ps"], c["cache"]
    b, pos = _positions(s)
    page = s["bt"][b, pos // ps].long()
    first = torch.full((s["kp"].shape[0],), ps, dtype=torch.long, device="cuda")
    first.scatter_reduce_(0, page, pos % ps, "amin")
    touched = (first < ps).nonzero().squeeze(1)
    old = (torch.arange(ps, device="cuda")[None, :] < first[touched, None])[:, None, :, None]
    for x, pages, scales in ((s["k"], s["kp"], s["ks"]), (s["v"], s["vp"], s["vs"])):
        amax = torch.zeros(scales.shape, device="cuda")
        amax.scatter_reduce_(0, page[:, None].expand(-1, hkv), x.float().abs().amax(2), "amax")
        m, e = torch.frexp(amax / QMAX[kind])
        need = torch.where(amax > 0, torch.exp2((e - (m == 0.5).int()).float()), 0.0)
        was = scales[touched] * (first[touched, None] > 0)
        now = torch.maximum(was, need[touched])
        safe = torch.where(now > 0, now, 1.0)
        vals = pages[touched].float() * (was / safe)[:, :, None, None]
        if kind == "int8":
            vals = vals.round()
        pages[touched] = torch.where(old, vals.to(pages.dtype).float(),
                                     pages[touched].float()).to(pages.dtype)
        scales[touched] = now
        y = x.float() / torch.where(scales > 0, scales, 1.0)[page][:, :, None]
        pages[page, :, pos % ps] = (y.round() if kind == "int8" else y).to(pages.dtype)
    return s["kp"], s["vp"], s["ks"], s["vs"]


def _touched(s):
    """(sequence, block) of every block that holds a new token."""
    bs = s["case"]["bs"]
    first = (s["used"].long() - (s["cu"][1:] - s["cu"][:-1])) // bs
    col = torch.arange(s["rows"].shape[1], device="cuda")[None, :]
    return ((col >= first[:, None]) & (col * bs < s["used"][:, None])).nonzero(as_tuple=True)


def _keys(s, b, blk):
    """Page ids [n, pages per block] of blocks and which keys [n, block] live."""
    c = s["case"]
    per = c["bs"] // c["ps"]
    pid = s["bt"][b[:, None], blk[:, None] * per + torch.arange(per, device="cuda")].long()
    at = blk[:, None] * c["bs"] + torch.arange(c["bs"], device="cuda")
    live = (at < s["used"][b][:, None]) & (pid >= 0).repeat_interleave(c["ps"], 1)
    return pid.clamp(min=0), live


def _bounds_plain(s, real=torch.float32):
    c = s["case"]
    b, blk = _touched(s)
    pid, live = _keys(s, b, blk)
    k = s["kp"][pid].to(real) * s["ks"][pid].to(real)[..., None, None]
    k = k.transpose(1, 2).reshape(len(b), c["hkv"], c["bs"], c["d"])
    dead = ~live[:, None, :, None]
    both = torch.stack([k.masked_fill(dead, math.inf).amin(2),
                        k.masked_fill(dead, -math.inf).amax(2)], 2)
    if real == torch.float64:
        out = s["bounds"].to(real)
        out[s["rows"][b, blk].long()] = both
        return out
    s["bounds"][s["rows"][b, blk].long()] = both.to(torch.bfloat16)
    return s["bounds"]


def _select_plain(s):
    """Scores in 64 bits: which block comes in may turn on the last bits."""
    c = s["case"]
    tq, hkv, d, bs, topk = s["q"].shape[0], c["hkv"], c["d"], c["bs"], c["topk"]
    b, pos = _positions(s)
    q = s["q"].double().view(tq, hkv, -1, d)
    pooled = torch.cat([q.clamp(max=0).sum(2), q.clamp(min=0).sum(2)], 2)      # [tq, hkv, 2 d]
    n = s["rows"].shape[1]
    # one product per (sequence, kv head), the queries padded to the longest sequence's
    t = torch.arange(tq, device="cuda") - s["cu"][b]
    wide = torch.zeros((c["batch"], int(np.diff(s["cu_host"]).max()), hkv, 2 * d),
                       dtype=torch.float64, device="cuda")
    wide[b, t] = pooled
    box = s["bounds"][s["rows"].long().clamp(min=0)].double().view(c["batch"], n, hkv, 2 * d)
    score = torch.einsum("bqhx,bnhx->bqhn", wide, box)[b, t]
    nblk = (pos // bs + 1)[:, None, None]
    col = torch.arange(n, device="cuda")
    score = score.masked_fill(col >= nblk, -math.inf)
    order = torch.sort(score, dim=2, descending=True, stable=True).indices[:, :, :topk]
    order = torch.where(order < nblk, order, n).sort(2).values
    out = torch.full((tq, hkv, topk), -1, dtype=torch.int32, device="cuda")
    out[:, :, :order.shape[2]] = torch.where(order < n, order, -1)
    return out


def _attend_plain(s, real=torch.float32, rows=None):
    """Gather the selected blocks' keys and values, softmax, weighted sum."""
    c = s["case"]
    hkv, d, bs = c["hkv"], c["d"], c["bs"]
    at = slice(None) if rows is None else rows
    sel = s["selected"][at].long()
    b, pos = (x[at] for x in _positions(s))
    tq, g = len(b), c["hq"] // hkv
    n = sel.shape[2]
    flat = sel.reshape(-1)
    bb = b[:, None, None].expand_as(sel).reshape(-1)
    pid, live = _keys(s, bb, flat.clamp(min=0))
    live &= (flat >= 0)[:, None]
    key = flat[:, None] * bs + torch.arange(bs, device="cuda")
    live &= key <= pos[:, None, None].expand_as(sel).reshape(-1)[:, None]
    live = live.view(tq, hkv, 1, n * bs)
    h = torch.arange(hkv, device="cuda")[None, :, None].expand_as(sel).reshape(-1)[:, None]

    def take(pages, scales):
        x = pages[pid, h].to(real) * scales[pid, h].to(real)[..., None, None]
        return x.view(tq, hkv, n * bs, d)

    q = s["q"][at].to(real).view(tq, hkv, g, d)
    w = (q @ take(s["kp"], s["ks"]).transpose(2, 3)) / math.sqrt(d)
    w = w.masked_fill(~live, -math.inf)
    top = w.amax(3, keepdim=True).clamp(min=-1e30)
    w = torch.exp(w - top)
    total = w.sum(3, keepdim=True)
    out = (w @ take(s["vp"], s["vs"])) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).view(tq, c["hq"])
    out = out.view(tq, c["hq"], d)
    return out, lse


# ----------------------------------------------------------------------------- runs

def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "store":
        return _store_plain(s)
    if c["op"] == "bounds":
        return _bounds_plain(s)
    if c["op"] == "select":
        return _select_plain(s)
    out, lse = _attend_plain(s)
    return out.to(s["q"].dtype), lse


def _run_own(s, c):
    import block_sparse_paged_csr_gb300 as sa

    kept = s["kept"]         # buffers that a serving loop keeps from step to step
    if c["op"] == "store":
        sa.sa_store_kv(s["k"], s["v"], s["kp"], s["vp"], s["bt"], s["cu_host"], s["cu"], s["used"],
                       k_scales=s["ks"], v_scales=s["vs"])
        return s["kp"], s["vp"], s["ks"], s["vs"]
    if c["op"] == "bounds":
        return sa.sa_block_bounds(s["kp"], s["bt"], s["cu_host"], s["cu"], s["used"], s["bounds"],
                                  s["rows"], c["bs"], k_scales=s["ks"])
    if c["op"] == "select":
        if not kept:
            kept["workspace"] = sa.allocate_select_workspace(
                s["q"].shape[0], c["batch"], c["hkv"], c["d"], s["rows"].shape[1], s["q"].device)
            kept["selected"] = torch.empty((s["q"].shape[0], c["hkv"], c["topk"]),
                                           dtype=torch.int32, device=s["q"].device)
        return sa.sa_select_blocks(s["q"], s["bounds"], s["rows"], s["cu_host"], s["cu"], s["used"],
                                   c["bs"], c["topk"], True, **kept)
    out, lse, index, partials = sa.sa_attention(
        s["q"], s["kp"], s["vp"], s["selected"], s["cu_host"], s["cu"], s["used"], s["bt"], c["hq"],
        c["hkv"], c["d"], c["bs"], c["ps"], 1.0 / math.sqrt(c["d"]), True, k_scales=s["ks"],
        v_scales=s["vs"], **kept)
    kept.update(index=index, partials=partials, out=out, lse=lse)
    return out, lse


# ----------------------------------------------------------------------------- work

def work(case):
    """Of one pass, lengths at their expected values."""
    c = case
    size = {"f32": 4, "bf16": 2}[c["act"]]
    qo = (c["qo_min"] + c["qo_max"]) / 2
    lk = max((c["kv_min"] + c["kv_max"]) / 2, qo)
    tq, hkv, d, bs = c["batch"] * qo, c["hkv"], c["d"], c["bs"]
    if c["op"] == "store":
        new = 2 * tq * hkv * d
        return {"bytes": new * (size + 1), "flops": 3 * new}
    if c["op"] == "bounds":
        blocks = c["batch"] * min(math.ceil(lk / bs), math.ceil(qo / bs) + (qo < lk))
        keys = c["batch"] * bs / 2 if qo == 1 else c["batch"] * qo
        return {"bytes": keys * hkv * d + blocks * hkv * 4 * d, "flops": 2 * keys * hkv * d}
    if c["op"] == "select":
        nblk = math.ceil(lk / bs)
        return {"bytes": tq * c["hq"] * d * size + c["batch"] * nblk * hkv * 4 * d
                + tq * hkv * c["topk"] * 4, "flops": 4 * tq * hkv * nblk * d}
    blocks = min(c["topk"], math.ceil(lk / bs))
    edges = tq * hkv * (1 + 0.9 * (blocks - 1))
    # each block of a sequence that is selected at all is read once
    read = min(edges, c["batch"] * hkv * math.ceil(lk / bs))
    return {"bytes": read * bs * 2 * d + 2 * tq * c["hq"] * d * size + tq * c["hq"] * 4,
            "flops": edges * (c["hq"] // hkv) * bs * 4 * d}


# ----------------------------------------------------------------------------- in 64 bits

def _store_exact(s):
    """Page by page from the definition, in numpy."""
    c = s["case"]
    ps, kind = c["ps"], c["cache"]
    lk, cu, bt = s["used"].cpu().numpy(), s["cu_host"], s["bt"].cpu().numpy()
    outs = []
    for x, pages, scales in ((s["k"], s["kp"], s["ks"]), (s["v"], s["vp"], s["vs"])):
        x = x.double().cpu().numpy()
        codes = pages.float().double().cpu().numpy()
        scales = scales.double().cpu().numpy()
        for b in range(len(lk)):
            start = int(lk[b] - (cu[b + 1] - cu[b]))
            at = start
            while at < lk[b]:
                r0, end = at % ps, min(int(lk[b]), (at // ps + 1) * ps)
                page = bt[b, at // ps]
                new = x[cu[b] + at - start:cu[b] + end - start]                 # [n, hkv, d]
                amax = np.abs(new).max(axis=(0, 2))
                with np.errstate(divide="ignore"):
                    need = np.where(amax > 0, 2.0 ** np.ceil(np.log2(amax / QMAX[kind])), 0.0)
                was = scales[page] if r0 else np.zeros_like(need)
                now = np.maximum(was, need)
                safe = np.where(now > 0, now, 1.0)
                ratio = (was / safe)[:, None, None]
                codes[page, :, :r0] = _nearest(codes[page, :, :r0] * ratio, kind)
                codes[page, :, r0:r0 + len(new)] = _nearest(
                    new.transpose(1, 0, 2) / safe[:, None, None], kind)
                scales[page] = now
                at = end
        outs.append((codes, scales))
    (k, ks), (v, vs) = outs
    if kind == "int8":
        k, v = k.astype(np.int8), v.astype(np.int8)
    return tuple(torch.from_numpy(np.ascontiguousarray(a)) for a in (k, v, ks, vs))


def _nearest(y, kind):
    """To the nearest code: steps of one, or of an eighth of the power of two
    below (2^-9 under 2^-6); ties to even."""
    if kind == "int8":
        return np.round(y)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.abs(y)))
    step = 2.0 ** (np.maximum(e, -6.0) - 3.0)
    return np.round(y / step) * step


def _select_exact(s):
    """Query rows a piece at a time: the larger of q lo and q hi in every
    channel, summed; then a rank by (score, lower block first)."""
    c = s["case"]
    hkv, d, bs, topk = c["hkv"], c["d"], c["bs"], c["topk"]
    b, pos = _positions(s)
    n = s["rows"].shape[1]
    if s["q"].shape[0] * c["hq"] * n > 2 ** 25:
        return None
    out = []
    for i in range(s["q"].shape[0]):
        seen = int(pos[i]) // bs + 1
        box = s["bounds"][s["rows"][b[i], :seen].long()].double()              # [seen, hkv, 2, d]
        q = s["q"][i].double().view(hkv, -1, d)
        best = torch.zeros((seen, hkv), dtype=torch.float64, device="cuda")
        for lane in range(q.shape[1]):
            best += (box * q[:, lane][None, :, None, :]).amax(2).sum(2)
        take = (-best).T.contiguous().cpu().numpy()
        row = np.full((hkv, topk), -1, np.int32)
        for h in range(hkv):
            ids = np.sort(np.lexsort((np.arange(seen), take[h]))[:topk])
            row[h, :len(ids)] = ids
        out.append(torch.from_numpy(row))
    return torch.stack(out)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "store":
        return _store_exact(s)
    if case["op"] == "bounds":
        return _bounds_plain(s, torch.float64)
    if case["op"] == "select":
        return _select_exact(s)
    # piece by piece: keys and values of a piece in 64 bits take up to 4 GB each
    c = case
    tq = s["q"].shape[0]
    step = max(1, (1 << 29) // (c["hkv"] * c["topk"] * c["bs"] * c["d"]))
    got = [_attend_exact(s, slice(at, min(at + step, tq))) for at in range(0, tq, step)]
    return torch.cat([g[0] for g in got]), torch.cat([g[1] for g in got])


def _attend_exact(s, rows):
    """Block by block with a running log-sum-exp, in 64 bits."""
    c = s["case"]
    hkv, d, bs, ps = c["hkv"], c["d"], c["bs"], c["ps"]
    sel = s["selected"][rows].long()
    b, pos = (x[rows] for x in _positions(s))
    q = s["q"][rows].double().view(len(b), hkv, -1, d) / math.sqrt(d)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    out = torch.zeros_like(q)
    h = torch.arange(hkv, device="cuda")
    for r in range(sel.shape[2]):
        for p in range(bs // ps):
            at = sel[:, :, r] * bs + p * ps                                    # [n, hkv]
            ok = (sel[:, :, r] >= 0) & (at < s["used"][b][:, None])
            page = s["bt"][b[:, None], (at // ps).clamp(0, s["bt"].shape[1] - 1)].long()
            page = page.clamp(min=0)
            key = at[:, :, None] + torch.arange(ps, device="cuda")
            ok = ok[:, :, None] & (key <= pos[:, None, None])
            k = s["kp"][page, h].double() * s["ks"][page, h].double()[..., None, None]
            v = s["vp"][page, h].double() * s["vs"][page, h].double()[..., None, None]
            w = torch.einsum("nhgd,nhkd->nhgk", q, k).masked_fill(~ok[:, :, None], -math.inf)
            new = torch.logaddexp(lse, torch.logsumexp(w, 3))
            safe = torch.where(new == -math.inf, 0.0, new)
            out = out * torch.exp(lse - safe)[..., None] + torch.einsum(
                "nhgk,nhkd->nhgd", torch.exp(w - safe[..., None]), v)
            lse = new
    return out.reshape(len(b), -1, d), lse.reshape(len(b), -1)
