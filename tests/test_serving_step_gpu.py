"""A serving loop of the operators together: projections are normalised and rotated,
stored, and attended over, densely and by selection; the cache is read back."""
import math

import numpy as np
import pytest
import torch

import block_sparse_paged_csr_gb300 as sa
from _serving import TORCH, f64, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,act", [("e4m3", "bf16"), ("int8", "f32"), ("bf16", "f32"), ("f32", "f32")])
def test_prompts_then_tokens(kind, act):
    """Prompts and then three tokens each: the dense attention over the cache is that of the
    rows that sa_load_kv reads back, the sparse attention over every block is the same, and
    the rows are what the norm and rotation make, up to the cache's type."""
    hq, hkv, d, ps, bs = 8, 2, 128, 16, 64
    lens = np.array([130, 64, 5, 300])
    cols = -(-(int(lens.max()) + 3) // bs) * (bs // ps)
    n = len(lens) * cols
    rng = np.random.default_rng(1)
    table = on_gpu(rng.permutation(n).reshape(len(lens), cols), np.int32)
    eight = kind in ("e4m3", "int8")
    pools = [torch.zeros((n, hkv, ps, d), device="cuda").to(TORCH[kind]) for _ in range(2)]
    scales = [torch.zeros((n, hkv), device="cuda") for _ in range(2)]
    kw = dict(k_scales=scales[0], v_scales=scales[1]) if eight else {}
    wq, wk = (1 + 0.1 * torch.randn((2, d), device="cuda")).to(TORCH[act])
    freq = on_gpu(10000.0 ** (-np.arange(d // 2) / (d // 2)), np.float32)
    status = torch.zeros(1, dtype=torch.int64, device="cuda")
    ws = sa.allocate_decode_workspace(len(lens), hq, hkv, d, "cuda")
    stored = [[] for _ in lens]
    for step in range(4):
        qo = lens if step == 0 else np.ones_like(lens)
        lk = lens + step
        cu = np.concatenate([[0], np.cumsum(qo)]).astype(np.int64)
        batch = (cu, on_gpu(cu, np.int64), on_gpu(lk, np.int32))
        q, k, v = torch.randn((int(cu[-1]), hq + 2 * hkv, d), device="cuda").to(TORCH[act]).split(
            (hq, hkv, hkv), 1)
        q, k = sa.sa_norm_rope(q, k, wq, wk, freq, cu_seqlens_q_host=cu, cu_seqlens_q=batch[1],
                               used_kv_lens=batch[2], status=status)
        sa.sa_store_kv(k, v, *pools, table, *batch, status=status, **kw)
        for b in range(len(lens)):
            stored[b].append((k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]]))
    out, lse = sa.sa_decode_attention(q, *pools, table, batch[2], 1 / math.sqrt(d), workspace=ws,
                                      status=status, **kw)
    whole = np.concatenate([[0], np.cumsum(lk)]).astype(np.int64)
    rk, rv = sa.sa_load_kv(*pools, table, whole, on_gpu(whole, np.int64), batch[2], dtype=torch.float32,
                           status=status, **kw)
    assert int(status) == 0
    for b in range(len(lens)):
        at = slice(whole[b], whole[b + 1])
        for got, which in ((rk[at], 0), (rv[at], 1)):
            made = torch.cat([s[which] for s in stored[b]]).float()
            # half a step of a code under the page's scale, whose largest magnitude may be up to twice
            # what fits it; a page that took a larger scale later rounds its codes once more: two
            # halves, 2 (2^-4, e4m3; 2^-7 of the range, int8); bf16 half a step
            tol = {"f32": 0.0, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -3, "int8": 2.0 ** -6}[kind]
            top = made.abs() if kind in ("f32", "bf16") else made.abs().amax()
            assert ((got - made).abs() <= tol * top).all()
        x = np.einsum("hgd,nhd->hgn", f64(q[b]).reshape(hkv, -1, d), f64(rk[at])) / math.sqrt(d)
        m = x.max(2, keepdims=True)
        p = np.exp(x - m)
        ref = np.einsum("hgn,nhd->hgd", p / p.sum(2, keepdims=True), f64(rv[at])).reshape(hq, d)
        tol = 2.0 ** -7 if act == "bf16" else 1e-5
        err = np.abs(f64(out[b]) - ref).max() / np.abs(ref).max()
        assert err <= tol, err
        rlse = (m[..., 0] + np.log(p.sum(2))).reshape(hq)
        assert np.abs(f64(lse[b]) - rlse).max() <= 1e-5 * np.abs(rlse).max()
    if act == "f32" or eight:
        sel = torch.arange(cols * ps // bs, dtype=torch.int32, device="cuda").repeat(len(lens), hkv, 1)
        sel = torch.where(sel * bs < batch[2][:, None, None], sel, -1)
        same, slse, index, _ = sa.sa_attention(q, *pools, sel, *batch, table, hq, hkv, d, bs, ps,
                                               1 / math.sqrt(d), True, **kw)
        assert sa.sa_get_status(index) == 0
        # (the sparse path over f32 queries and bf16 keys splits its operands into 16 bits)
        torch.testing.assert_close(out.float(), same.float(), rtol=2.0 ** -7 if act == "bf16" else 1e-4,
                                   atol=1e-2 if act == "bf16" else 1e-4)
        torch.testing.assert_close(lse, slse, rtol=1e-4, atol=1e-4)


def test_one_graph_for_a_step():
    """Norm, rotation, store and attention captured together and replayed as the sequences
    grow."""
    hq, hkv, d, ps, b = 4, 1, 64, 16, 3
    table = torch.arange(b * 4, dtype=torch.int32, device="cuda").view(b, 4)
    pools = [torch.zeros((b * 4, hkv, ps, d), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    freq = on_gpu(10000.0 ** (-np.arange(32) / 32), np.float32)
    w = torch.ones(d, device="cuda")
    cu = np.arange(b + 1)
    cud, used = on_gpu(cu, np.int64), on_gpu([1, 20, 0], np.int32)
    qkv = torch.randn((b, hq + 2 * hkv, d), device="cuda")
    ws = sa.allocate_decode_workspace(b, hq, hkv, d, "cuda")
    out, lse = torch.empty((b, hq, d), device="cuda"), torch.empty((b, hq), device="cuda")
    qr, kr = torch.empty((b, hq, d), device="cuda"), torch.empty((b, hkv, d), device="cuda")

    def step(out, lse, qr, kr, pools):
        q, k, v = qkv.split((hq, hkv, hkv), 1)
        sa.sa_norm_rope(q, k, w, w, freq, cu_seqlens_q_host=cu, cu_seqlens_q=cud, used_kv_lens=used,
                        q_out=qr, k_out=kr)
        sa.sa_store_kv(kr, v, *pools, table, cu, cud, used)
        sa.sa_decode_attention(qr, *pools, table, used, 0.125, out=out, lse=lse, workspace=ws)

    eager = [torch.empty_like(t) for t in (out, lse, qr, kr)]
    mine = [p.clone() for p in pools]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(out, lse, qr, kr, pools)
    for _ in range(5):
        qkv.normal_()
        g.replay()
        step(*eager, mine)
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1]) and torch.equal(kr, eager[3])
        used += 1
    assert torch.equal(pools[0], mine[0]) and torch.equal(pools[1], mine[1])
