"""How many bits sa_decode_attention keeps, where its outputs would hide a loss of them."""
import math

import numpy as np
import pytest
import torch

import block_sparse_paged_csr_gb300 as sa
from _serving import TORCH

pytestmark = pytest.mark.gpu
KINDS = ["f32", "bf16", "e4m3", "int8"]
U = 2.0 ** -24


def pools(shape, kind, gen, spread=40.0):
    """Random K and V pools, their scales' arguments, and their values in 64 bits."""
    pages, values, kw = [], [], {}
    for name in ("k_scales", "v_scales"):
        x = torch.randn(shape, generator=gen, device="cuda")
        if kind == "int8":
            x = (x * spread).round().clamp(-127, 127)
        elif kind == "e4m3":
            x = (x * 2 * spread).clamp(-448, 448)
        x = x.to(TORCH[kind])
        v = x.float().double()
        if kind in ("int8", "e4m3"):
            s = torch.exp2(torch.randint(-7, -4, shape[:2], generator=gen, device="cuda").float())
            kw[name] = s
            v = v * s.double()[:, :, None, None]
        pages.append(x)
        values.append(v)
    return pages, values, kw


def half_step(x):
    """Half of the distance of bf16 numbers at magnitudes x (8 bits)."""
    return torch.exp2(torch.floor(torch.log2(x.clamp(min=1e-30))) - 8)


@pytest.mark.parametrize("g", [4, 12])
@pytest.mark.parametrize("kind", KINDS)
def test_bf16_outputs_are_the_formulas_rounded_once(kind, g):
    """bf16 queries: what comes out is the formula's value rounded once, but for the f32 arithmetic
    before it.  Three keys a sequence (one tile, no merges) with scores near 0, so that this arithmetic
    is known closely: a score of at most big = sum |q k| scale is off by 2 (d + 16) 2^-24 big (d
    roundings, 16 more for operands in parts, doubled for the tensor cores' cuts) and 3 2^-24 in base 2;
    numerator and denominator have it both, with 2^-22 of ex2; P's parts and V's (f32) leave 2^-21
    each, sums and the quotient some 10 roundings.  All of it relative to sum p |v|: signs that cancel make it
    large beside the output's own half step."""
    n, d, hkv, batch = 3, 64, 4, 1500
    gen = torch.Generator(device="cuda").manual_seed(g)
    (kp, vp), (k, v), kw = pools((batch, hkv, n, d), kind, gen)
    q = (0.002 * torch.randn((batch, hkv * g, d), generator=gen, device="cuda")).bfloat16()
    table = torch.randperm(batch, generator=gen, device="cuda").to(torch.int32)[:, None].contiguous()
    used = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    out, _ = sa.sa_decode_attention(q, kp, vp, table, used, 0.125, **kw)
    at = table[:, 0].long()
    x = q.double().view(batch, hkv, g, d) * 0.125
    big = float((x.abs() @ k[at].abs().transpose(2, 3)).max())
    p = torch.softmax(x @ k[at].transpose(2, 3), 3)
    ref, size = p @ v[at], p @ v[at].abs()
    part = 2 * (2 * (d + 16) * U * big + 3 * U) + 2 * 2.0 ** -22 + 2 * 2.0 ** -21 + 10 * U
    assert part < 2.0 ** -18
    off = part * size
    err = (out.double().view_as(ref) - ref).abs()
    wrong = int((~(err <= off + half_step(ref.abs() + off))).sum())
    assert wrong == 0, f"{wrong} of {err.numel()}"


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("g", [4, 12])
@pytest.mark.parametrize("kind", KINDS)
def test_a_key_that_takes_nearly_all_leaves_the_others_their_bits(kind, g, act):
    """One key among 32768 holds all but some 2^-13 of the softmax, its V row is 0 (and shares its page
    with ordinary rows), so that the output is the others' alone: products of 2^-28 of the largest.
    Tolerance, relative to their sum p |v|: twice the scores' errors (theirs are small; the large one's
    is common to all in l: 2 (d + 16) 2^-24 of its size), and over 8 bits the parts' last unit: the
    remainder of a product keeps 2^-36 of a unit of which the largest counts 2^3 or more, 2^-39 of the
    largest P vs a key, times its code.  These roundings are independent: their sum over the keys has
    a deviation below sqrt(n) 2^-39 128 (448) and is taken six times.  (In f16 without the remainders'
    own scale 2^-28 a key: that is as large as the products.)"""
    n, d, hkv, ps, batch = 32768, 64, 2, 64, 1300
    gen = torch.Generator(device="cuda").manual_seed(g)
    (kp, vp), _, kw = pools((n // ps, hkv, ps, d), kind, gen)
    for name in kw:
        kw[name].fill_(2.0 ** -6)
    # channel 0 is the large key's: 8 in the queries, 1 in its row, 0 in the other keys'
    page, row = 11, 37
    kp.view(torch.uint8).view(*kp.shape, -1)[..., 0, :] = 0
    key = torch.zeros((hkv, d), device="cuda")
    key[:, 0] = 64.0 if kw else 1.0
    kp[page, :, row] = key.to(TORCH[kind])
    vp[page, :, row] = torch.zeros((hkv, d), device="cuda").to(TORCH[kind])
    scale = (math.log(n) + 13 * math.log(2.0)) / 8.0        # its score: 19.4
    q = torch.randn((batch, hkv * g, d), generator=gen, device="cuda") * 0.1 / scale
    q[..., 0] = 8.0                                         # (the others' scores: some 0.1 sqrt(d))
    q = q.to(TORCH[act])
    # (the sequences share their pages, so that a warp has the large key and many others in one piece)
    table = torch.randperm(n // ps, generator=gen, device="cuda").to(torch.int32).repeat(batch, 1)
    used = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    out, _ = sa.sa_decode_attention(q, kp, vp, table, used, scale, **kw)
    kk, vv = ((x.float().double() * (2.0 ** -6 if kw else 1)).transpose(0, 1).reshape(hkv, n, d) for x in (kp, vp))
    for b in range(0, batch, 29):
        x = q[b].double().view(hkv, g, d) * scale
        p = torch.softmax(x @ kk.transpose(1, 2), 2)
        ref, size = p @ vv, p @ vv.abs()
        held = p[:, :, page * ps + row]
        assert 2.0 ** -15 < float((1 - held).min()) and float((1 - held).max()) < 2.0 ** -11
        big = (x.abs() @ kk.abs().transpose(1, 2)).amax(2)[..., None]
        tol = (2 * 2 * (d + 16) * U * (big + 1) + 3 * U * (big + 1)) * size
        if kw:
            tol = tol + 6 * math.sqrt(n) * 2.0 ** -39 * held[..., None] * 2.0 ** -6 * (
                128 if kind == "int8" else 448)
        # what the tolerance leaves of the others' part
        assert float((tol / size).median()) < 2.0 ** -8
        if act == "bf16":
            tol = tol + half_step(ref.abs() + tol)
        err = (out[b].double().view_as(ref) - ref).abs()
        worst = float((err / tol).nan_to_num(nan=math.inf).max())
        assert worst <= 1


@pytest.mark.parametrize("kind", KINDS)
def test_long_sums_of_bf16_queries_do_not_drift(kind):
    """Sums over many tiles by one warp, 1024 sequences of 65536 keys that share their pages: at least
    1700 tiles of 32 keys a warp.  Sums that are cut at every step of 16 keys would leave 3400 2^-26 =
    5e-5 of the output missing.  Values near 1.5 and scores wide enough (some 100 keys count) that the
    outputs spread over several steps of bf16: their roundings, at most 2^-8 / sqrt(3) of deviation,
    vanish in the mean over 2^18 outputs to 4.4e-6, of which five are allowed, and 1e-6 for the
    rest (a tile's own products are cut at most 3 times 2^-24, ex2 2^-22 on both sides)."""
    batch, hkv, g, n, d, ps = 1024, 2, 2, 65536, 64, 64
    gen = torch.Generator(device="cuda").manual_seed(5)
    shape = (n // ps, hkv, ps, d)
    k = torch.randn(shape, generator=gen, device="cuda")
    v = 1.5 + 0.4 * torch.randn(shape, generator=gen, device="cuda")
    kw = {}
    if kind in ("e4m3", "int8"):
        k, v = (k * 30).to(TORCH[kind]), (v.clamp(0, 3.9) * 32).to(TORCH[kind])
        s = torch.full((n // ps, hkv), 2.0 ** -5, device="cuda")
        kw = dict(k_scales=s, v_scales=s)
    else:
        k, v = k.to(TORCH[kind]), v.to(TORCH[kind])
    kx, vx = (x.float().double() * (2.0 ** -5 if kw else 1) for x in (k, v))
    table = torch.arange(n // ps, dtype=torch.int32, device="cuda").repeat(batch, 1)
    q = (2.5 * torch.randn((batch, hkv * g, d), generator=gen, device="cuda")).bfloat16()
    used = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    out, _ = sa.sa_decode_attention(q, k, v, table, used, 0.125, **kw)
    off = []
    for h in range(hkv):
        keys, vals = (x[:, h].reshape(n, d) for x in (kx, vx))
        for rows in q[:, h * g:(h + 1) * g].double().reshape(-1, d).split(512):
            off.append(torch.softmax(rows @ keys.T * 0.125, 1) @ vals)
    ref = torch.stack([x for x in torch.cat(off).view(hkv, batch, g, d)], 1).reshape(batch, hkv * g, d)
    # (roundings of a normal spread of s steps have a mean of exp(-2 pi^2 s^2) / pi steps at most: with two
    # steps nothing)
    assert float(ref.std()) > 2 * 2.0 ** -7
    mean = float(((out.double() - ref) / ref).mean())
    assert abs(mean) <= 1e-6 + 5 * 2.0 ** -8 / math.sqrt(3 * ref.numel()), mean
