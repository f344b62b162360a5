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
@pytest.mark.parametrize("kind", ["f32", "e4m3", "int8"])
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
