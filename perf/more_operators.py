"""What the measurements of the operators around a paged cache run.

Three operators of a serving step that stand beside storing, selecting and sparse attention:
queries and keys are normalised per head and rotated by their positions (``rope``), one new
token of each sequence attends over its whole cache or a window of it (``decode``), and rows
of the cache are read back as they were stored (``load``).

``own`` False computes each operator in plain torch; True calls the library.
"""
import math

import numpy as np
import torch

own = False

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
         "int8": torch.int8}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1, "int8": 1}
EPS = 1e-6
BASE = 500000.0          # of the rotation's frequencies


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of each of 64 running sequences: what a decode step does first (latency)
        dict(name="rope_decode", op="rope", batch=64, qo_min=1, qo_max=1, kv_min=300, kv_max=2000,
             hq=32, hkv=8, d=128, rot=128, axes=1, pairs="halves", norm=True, act="bf16",
             out="bf16"),
        # the chunk of a chunked prefill, f32 activations
        dict(name="rope_prompt", op="rope", batch=4, qo_min=2048, qo_max=2048, kv_min=32768,
             kv_max=32768, hq=64, hkv=8, d=128, rot=128, axes=1, pairs="halves", norm=True,
             act="f32", out="f32"),
        # prompts with images: positions of time, height and width, half of a head rotated in
        # adjacent pairs; f32 out, which attention over f32 and bf16 caches takes
        dict(name="rope_axes", op="rope", batch=3, qo_min=900, qo_max=1700, kv_min=1700,
             kv_max=5000, hq=28, hkv=4, d=128, rot=64, axes=3, pairs="adjacent", norm=True,
             act="bf16", out="f32"),
        # a few short sequences, one of them a padding row of length 0, small odd heads: latency
        dict(name="decode_small", op="decode", batch=4, kv_min=0, kv_max=700, hq=6, hkv=2, d=64,
             ps=16, window=0, cache="int8", act="f32"),
        # the grouped-query decode batch over a bf16 cache
        dict(name="decode_gqa", op="decode", batch=64, kv_min=4096, kv_max=32768, hq=32, hkv=8,
             d=128, ps=16, window=0, cache="bf16", act="f32"),
        # one long conversation alone: its cache has to be split over the whole GPU
        dict(name="decode_one", op="decode", batch=1, kv_min=131072, kv_max=131072, hq=64, hkv=8,
             d=128, ps=64, window=0, cache="int8", act="bf16"),
        # a small batch over an f32 cache
        dict(name="decode_f32", op="decode", batch=16, kv_min=1000, kv_max=6000, hq=32, hkv=8,
             d=128, ps=16, window=0, cache="f32", act="f32"),
        # long contexts of many sequences in 8 bits
        dict(name="decode_long", op="decode", batch=64, kv_min=20000, kv_max=50000, hq=64, hkv=8,
             d=128, ps=16, window=0, cache="e4m3", act="bf16"),
        # a sliding-window layer with wide heads
        dict(name="decode_window", op="decode", batch=48, kv_min=2000, kv_max=60000, hq=16, hkv=2,
             d=256, ps=32, window=4096, cache="bf16", act="bf16"),
        # the prefixes of a few short sequences read back (latency)
        dict(name="load_small", op="load", batch=8, qo_min=20, qo_max=300, kv_min=300, kv_max=600,
             hq=32, hkv=8, d=128, ps=16, cache="int8", out="bf16"),
        # whole long prompts out of an 8-bit cache
        dict(name="load_prompt", op="load", batch=4, qo_min=20001, qo_max=32768, kv_min=32768,
             kv_max=32768, hq=64, hkv=8, d=128, ps=64, cache="e4m3", out="bf16"),
        # a chunk of four sequences out of a bf16 cache into f32
        dict(name="load_chunk", op="load", batch=4, qo_min=1501, qo_max=2048, kv_min=4096,
             kv_max=8192, hq=16, hkv=4, d=256, ps=32, cache="bf16", out="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "decode", "decode", "load"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 128, 128, 128, 256, 96, 80])
    c = dict(op=op, hkv=hkv, hq=hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), d=d)
    act = rng.choice(["f32", "bf16"])
    kind = rng.choice(["f32", "bf16", "e4m3", "int8"])
    if op == "decode":
        batch = _log(rng, 1, 100)
        kv = [_log(rng, 1, 30000) for _ in range(2)]
        c.update(batch=batch, kv_min=min(kv), kv_max=max(kv), ps=rng.choice([8, 16, 16, 32, 64]),
                 window=rng.choice([0, 0, _log(rng, 30, 8000)]), cache=kind, act=act)
        # rows x keys x channels of the padded cache in 32 bits stay below 13 GB
        while c["batch"] * c["kv_max"] * hkv * d > 2 ** 31 + 2 ** 30:
            c["batch"] = max(1, c["batch"] // 2)
        return c
    decode = rng.random() < 0.3
    qo = 1 if decode else _log(rng, 2, 6000)
    c.update(batch=_log(rng, 1, 100) if decode else rng.randint(1, 4),
             qo_min=1 if decode else max(1, qo // 2), qo_max=qo, kv_min=qo, kv_max=qo + 2000)
    if op == "rope":
        c.update(rot=rng.choice([d, d, d // 2]), axes=rng.choice([1, 1, 2, 3]),
                 pairs=rng.choice(["halves", "adjacent"]), norm=rng.random() < 0.8, act=act,
                 out=rng.choice([act, "f32"]))
    else:
        c.update(ps=rng.choice([8, 16, 32, 64]), cache=kind, out=rng.choice(["f32", "bf16"]))
    return c


# ----------------------------------------------------------------------------- inputs

def _lengths(case, seed):
    """Rows asked for and length of every sequence: of the case's own making, in the seed's
    order, so that the outputs of every seed have the same shapes."""
    rng = np.random.default_rng(case["batch"] + case["kv_max"])
    qo = rng.integers(case.get("qo_min", 1), case.get("qo_max", 1) + 1, case["batch"])
    lk = rng.integers(case["kv_min"], case["kv_max"] + 1, case["batch"])
    if case["op"] != "decode":
        lk = np.maximum(lk, qo)
    elif case["kv_min"] == 0:
        lk[0] = 0                # a padding row
    order = np.random.default_rng(seed).permutation(len(qo))
    return qo[order].astype(np.int64), lk[order].astype(np.int32)


def _tables(lk, per, gen):
    """[batch, columns] table of a randomly permuted pool with just the entries the lengths
    need (-1 behind them), and the pool's size."""
    live = torch.from_numpy(-(-lk.astype(np.int64) // per))
    cols = max(int(live.max()), 1)
    there = torch.arange(cols)[None, :] < live[:, None]
    n = max(int(live.sum()), 1)
    t = torch.full((len(lk), cols), -1, dtype=torch.int32, device="cuda")
    t[there.cuda()] = torch.randperm(n, generator=gen, device="cuda")[:int(live.sum())].to(torch.int32)
    return t, n


def _pool(shape, kind, gen):
    """Normal values (codes in 8 bits), made 2^28 elements at a time."""
    out = torch.empty(shape, dtype=TORCH[kind], device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for at in range(0, flat.numel(), step):
        x = torch.randn(min(step, flat.numel() - at), generator=gen, device="cuda")
        if kind == "int8":
            x = x.mul_(28.0).round_().clamp_(-127, 127)
        elif kind == "e4m3":
            x = x.mul_(96.0).clamp_(-448, 448)
        flat[at:at + step] = x.to(TORCH[kind])
    return out


def _scales(shape, kind, gen):
    """Powers of two, as the store makes them."""
    e = torch.randint(-6, -3, shape, generator=gen, device="cuda")
    return torch.exp2((e if kind == "int8" else e - 2).float())


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = case
    qo, lk = _lengths(c, seed)
    cu = np.concatenate([[0], np.cumsum(qo)]).astype(np.int64)
    tq, hq, hkv, d = int(cu[-1]), c["hq"], c["hkv"], c["d"]
    s = dict(case=c, cu_host=cu, cu=torch.from_numpy(cu).cuda(), used=torch.from_numpy(lk).cuda(),
             kept={})
    if c["op"] == "rope":
        # heads as a fused projection leaves them: q and k are slices of one tensor
        qkv = torch.randn((tq, hq + 2 * hkv, d), generator=gen, device="cuda")
        qkv *= torch.exp(0.5 * torch.randn((hq + 2 * hkv, d), generator=gen, device="cuda"))
        qkv = qkv.to(TORCH[c["act"]])
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        if c["norm"]:
            s["wq"], s["wk"] = (1 + 0.2 * torch.randn((2, d), generator=gen, device="cuda")).to(
                TORCH[c["act"]])
        else:
            s["wq"] = s["wk"] = None
        n = c["rot"] // 2
        s["freq"] = (BASE ** (-torch.arange(n, dtype=torch.float64) / n)).float().cuda()
        s["pos"] = s["axes"] = None
        if c["axes"] > 1:
            # a picture's patches in rows of 37: its place in time for all, then row and column
            _, p = _positions(s)
            at = torch.stack([p // 1000, p % 1000 // 37, p % 37])[:c["axes"]]
            s["pos"] = (at + torch.randint(0, 4000, (c["axes"], 1), generator=gen,
                                           device="cuda")).to(torch.int32)
            s["axes"] = (torch.arange(n, device="cuda") % c["axes"]).to(torch.int32)
        return s
    s["bt"], n = _tables(lk, c["ps"], gen)
    shape = (n, hkv, c["ps"], d)
    s["kp"], s["vp"] = _pool(shape, c["cache"], gen), _pool(shape, c["cache"], gen)
    s["ks"] = s["vs"] = None
    if SIZE[c["cache"]] == 1:
        s["ks"], s["vs"] = (_scales((n, hkv), c["cache"], gen) for _ in range(2))
    if c["op"] == "decode":
        s["q"] = torch.randn((c["batch"], hq, d), generator=gen, device="cuda").to(TORCH[c["act"]])
    return s


def _positions(s):
    """Sequence and position in it of every new token: the last ones of its sequence."""
    cu, used = s["cu"], s["used"].long()
    i = torch.arange(int(s["cu_host"][-1]), device="cuda")
    b = torch.searchsorted(cu, i, right=True) - 1
    return b, used[b] - (cu[b + 1] - cu[b]) + i - cu[b]


# ----------------------------------------------------------------------------- plain forms

def _rope_plain(s):
    """Norm, then a rotation by angles that are made in 64 bits (positions times frequencies
    pass what 32 bits resolve)."""
    c = s["case"]
    rot = c["rot"]
    if s["pos"] is None:
        p = _positions(s)[1][:, None]
    else:
        p = s["pos"][s["axes"].long()].T
    angle = p.double() * s["freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) * w.float()
        r, rest = x[..., :rot], x[..., rot:]
        if c["pairs"] == "halves":
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat([a * cos - b * sin, a * sin + b * cos], 2)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, a * sin + b * cos], 3).flatten(2)
        return torch.cat([r, rest], 2).to(TORCH[c["out"]])

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _decode_plain(s):
    """All keys in sight of the longest sequence side by side, softmax, weighted sum."""
    c = s["case"]
    ps, d, hkv, window = c["ps"], c["d"], c["hkv"], c["window"]
    used = s["used"].long()
    n = max(s["bt"].shape[1] * ps, 1)
    n = min(n, window) if window else n
    first = (used - window).clamp(min=0) if window else torch.zeros_like(used)
    at = first[:, None] + torch.arange(n, device="cuda")                       # [b, n]
    live = at < used[:, None]
    page = torch.gather(s["bt"], 1, (at // ps).clamp(max=s["bt"].shape[1] - 1)).long().clamp(min=0)

    def take(pages, scales):
        x = pages.transpose(1, 2)[page, at % ps].float()                       # [b, n, hkv, d]
        if scales is not None:
            x *= scales[page][..., None]
        return x.transpose(1, 2)

    q = s["q"].float().view(c["batch"], hkv, -1, d)
    w = (q @ take(s["kp"], s["ks"]).transpose(2, 3)) / math.sqrt(d)
    w = w.masked_fill(~live[:, None, None], -math.inf)
    top = w.amax(3, keepdim=True).clamp(min=-1e30)
    w = torch.exp(w - top)
    total = w.sum(3, keepdim=True)
    out = (w @ take(s["vp"], s["vs"])) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).view(c["batch"], -1)
    return out.view(c["batch"], -1, d).to(s["q"].dtype), lse


def _load_plain(s):
    c = s["case"]
    b, pos = _positions(s)
    page, row = s["bt"][b, pos // c["ps"]].long(), pos % c["ps"]

    def take(pages, scales):
        x = pages[page, :, row].float()
        if scales is not None:
            x = x * scales[page][:, :, None]
        return x.to(TORCH[c["out"]])

    return take(s["kp"], s["ks"]), take(s["vp"], s["vs"])


# ----------------------------------------------------------------------------- runs

def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "rope":
        return _rope_plain(s)
    return _decode_plain(s) if c["op"] == "decode" else _load_plain(s)


def _run_own(s, c):
    import block_sparse_paged_csr_gb300 as sa

    kept = s["kept"]         # buffers that a serving loop keeps from step to step
    if c["op"] == "rope":
        q, k = sa.sa_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["freq"], positions=s["pos"],
                               cu_seqlens_q_host=s["cu_host"], cu_seqlens_q=s["cu"],
                               used_kv_lens=s["used"], eps=EPS, freq_axes=s["axes"],
                               interleaved=c["pairs"] == "adjacent", out_dtype=TORCH[c["out"]],
                               **kept)
        kept.update(q_out=q, k_out=k)
        return q, k
    if c["op"] == "decode":
        if not kept:
            kept["workspace"] = sa.allocate_decode_workspace(c["batch"], c["hq"], c["hkv"], c["d"],
                                                             s["q"].device)
        out, lse = sa.sa_decode_attention(s["q"], s["kp"], s["vp"], s["bt"], s["used"],
                                          1.0 / math.sqrt(c["d"]), window=c["window"],
                                          k_scales=s["ks"], v_scales=s["vs"], **kept)
        kept.update(out=out, lse=lse)
        return out, lse
    k, v = sa.sa_load_kv(s["kp"], s["vp"], s["bt"], s["cu_host"], s["cu"], s["used"],
                         dtype=TORCH[c["out"]], k_scales=s["ks"], v_scales=s["vs"], **kept)
    kept.update(k=k, v=v)
    return k, v


# ----------------------------------------------------------------------------- work

def work(case):
    """Of one pass."""
    c = case
    qo, lk = _lengths(c, 0)
    tq, hkv, d = int(qo.sum()), c["hkv"], c["d"]
    if c["op"] == "rope":
        n = tq * (c["hq"] + hkv) * d
        return {"bytes": n * (SIZE[c["act"]] + SIZE[c["out"]]), "flops": 7 * n}
    if c["op"] == "load":
        n = 2 * tq * hkv * d
        return {"bytes": n * (SIZE[c["cache"]] + SIZE[c["out"]]), "flops": n}
    keys = int(np.minimum(lk, c["window"]).sum() if c["window"] else lk.sum())
    return {"bytes": keys * hkv * 2 * d * SIZE[c["cache"]]
            + c["batch"] * c["hq"] * (2 * d * SIZE[c["act"]] + 4),
            "flops": 4 * keys * c["hq"] * d}


# ----------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _rope_exact, "decode": _decode_exact, "load": _load_exact}[case["op"]](s)


def _rope_exact(s):
    """Pairs as complex numbers, turned by a product with a unit number."""
    c = s["case"]
    n = c["rot"] // 2
    if s["pos"] is None:
        cu, lk = s["cu_host"], s["used"].cpu().numpy()
        p = np.concatenate([np.arange(lk[b] - (cu[b + 1] - cu[b]), lk[b]) for b in range(len(lk))])
        p = np.repeat(p[:, None], n, 1)
    else:
        p = s["pos"].cpu().numpy()[s["axes"].cpu().numpy()].T
    turn = torch.polar(torch.ones(p.shape, dtype=torch.float64, device="cuda"),
                       torch.from_numpy(p.astype(np.float64)).cuda() * s["freq"].double())
    outs = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.double()
        if w is not None:
            size = torch.linalg.vector_norm(x, dim=2, keepdim=True)
            x = x * w.double() / torch.sqrt(size ** 2 / c["d"] + EPS)
        first = torch.arange(n, device="cuda") * (1 if c["pairs"] == "halves" else 2)
        other = first + (n if c["pairs"] == "halves" else 1)
        z = torch.complex(x[..., first], x[..., other]) * turn[:, None]
        x = x.clone()
        x[..., first], x[..., other] = z.real, z.imag
        outs.append(x)
    return tuple(outs)


def _rows(s, b, at):
    """Keys and values [hkv, n, d] in 64 bits of positions of sequence b."""
    c = s["case"]
    page = s["bt"][b, at // c["ps"]].long()
    got = []
    for pages, scales in ((s["kp"], s["ks"]), (s["vp"], s["vs"])):
        x = pages.flatten(0, 2).view(-1, c["d"])
        row = (page[:, None] * c["hkv"] + torch.arange(c["hkv"], device="cuda")) * c["ps"]
        x = x[row + (at % c["ps"])[:, None]].double()
        if scales is not None:
            x = x * scales.double()[page][:, :, None]
        got.append(x.transpose(0, 1))
    return got


def _decode_exact(s):
    """Sequence by sequence, the softmax by its logarithm."""
    c = s["case"]
    out = torch.zeros((c["batch"], c["hkv"], c["hq"] // c["hkv"], c["d"]), dtype=torch.float64,
                      device="cuda")
    lse = torch.full(out.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["used"].tolist()):
        if n == 0:
            continue
        at = torch.arange(max(0, n - c["window"]) if c["window"] else 0, n, device="cuda")
        k, v = _rows(s, b, at)
        q = s["q"][b].double().view(c["hkv"], -1, c["d"]) * c["d"] ** -0.5
        x = torch.einsum("hgd,hnd->hgn", q, k)
        lse[b] = torch.logsumexp(x, 2)
        out[b] = torch.einsum("hgn,hnd->hgd", torch.exp(x - lse[b][..., None]), v)
    return out.flatten(1, 2), lse.flatten(1)


def _load_exact(s):
    cu, got = s["cu_host"], []
    for b, n in enumerate(s["used"].tolist()):
        k, v = _rows(s, b, torch.arange(n - int(cu[b + 1] - cu[b]), n, device="cuda"))
        got.append((k.transpose(0, 1), v.transpose(0, 1)))
    return torch.cat([g[0] for g in got]), torch.cat([g[1] for g in got])
