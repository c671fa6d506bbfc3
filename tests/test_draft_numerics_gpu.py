"""Numerics of the drafted-decoding calls at the far ends of their ranges.  References and bounds
as in test_draft_gpu.
"""
import numpy as np
import pytest
import torch

import draft_ref as R
from test_draft_gpu import check_tree, ints, run_tree, tts  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# Cache rows
# ---------------------------------------------------------------------------
def far_rows(d):
    """Rows with entries so far below their largest that the quotient underflows, of both signs,
    each beside one that has to be decided exactly (a quotient below 2^-6)."""
    rows = []
    for top in (900.0, 1e10, 1e30, 3e38):
        for tiny in (2.0 ** -149, 2.0 ** -133, 1e-40, 1e-38, 2.0 ** -126, 1e-30):
            s = top / 448.0
            block = [top, 0.005 * s, -tiny, tiny, -0.0, 0.0, -0.0011 * s, -3 * tiny]
            rows.append((block * (d // 8))[:d])
    return np.array(rows, np.float64).astype(np.float32)


@pytest.mark.parametrize("kv", ["e4m3", "i8"])
@pytest.mark.parametrize("src", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_entries_far_below_their_row(tts, kv, src, d):  # noqa: F811
    g = np.random.default_rng(d)
    wide = (np.exp2(g.uniform(-149, 127, (500, d))) * g.choice([-1, 1], (500, d))).astype(np.float32)
    x = torch.from_numpy(np.concatenate([far_rows(d), wide])).to(R.TORCH[src])
    n = x.shape[0]
    c = R.Cache(1, 1, d, 1024, kv, 0, seed=2).to_device(tts, 2)
    rows = x.cuda()
    tts.tts_kv_write_rows(rows, rows, c.cache, c.desc, ints([0]), n)
    code, scale = R.to_cache(x.float().numpy(), kv)
    for t, s in ((c.dk, c.dks), (c.dv, c.dvs)):
        assert torch.equal(s[0, 0, :n].cpu(), scale)
        assert torch.equal(t[0, 0, :n].cpu().float(), code.float())   # (zeros of either sign are equal, NaN is not)


# ---------------------------------------------------------------------------
# Attention: softmax rows with one dominant entry
# ---------------------------------------------------------------------------
def seen(past, nodes, m, T):
    """Which positions node t sees, [T][past + nodes] (m: T masks as integers, or None)."""
    see = torch.zeros(T, past + nodes, dtype=torch.bool)
    see[:, :past] = True
    for t in range(nodes):
        bits = (2 << t) - 1 if m is None else int(m[t]) & ((1 << 64) - 1)
        for u in range(nodes):
            see[t, past + u] = bool(bits >> u & 1)
    return see


def attend(c, q, past, nodes, m, scale, b=0):
    """Stream b: q [T, Hq, D] f64 -> (out, mean |v|), as draft_ref.tree_attn, in one product."""
    n, grp = past + nodes, q.shape[1] // c.hkv
    K, V = (c.rows(w, b, n).repeat_interleave(grp, 1) for w in ("k", "v"))
    x = torch.einsum("thd,nhd->htn", q, K) * scale
    w = torch.softmax(x.masked_fill(~seen(past, nodes, m, q.shape[0]), -float("inf")), -1)
    return torch.einsum("htn,nhd->thd", w, V), torch.einsum("htn,nhd->thd", w, V.abs())


@pytest.mark.parametrize("kv", ["e4m3", "i8"])
@pytest.mark.parametrize("T", [1, 16, 64])
@pytest.mark.parametrize("n,small", [(4000, 0.1), (4000, 0.02), (16384, 0.02)])
def test_a_dominant_row_with_small_values(tts, kv, T, n, small):  # noqa: F811
    """One row takes 0.983 of the softmax and its V is small beside the others', which share the
    rest: each of their weights is 2^-18 to 2^-20 of the largest, all of them together half the
    output or more."""
    hq, hkv, d, B = 2, 1, 128, 40            # (streams enough that a CTA has long pieces of a window)
    g = np.random.default_rng(n + T)
    k = 0.01 * g.standard_normal((1, hkv, n, d)).astype(np.float32)
    v = np.abs(g.standard_normal((1, hkv, n, d))).astype(np.float32)
    top = np.log(0.983 / 0.017 * n)          # the dominant row's score above the others' (near 0)
    k[0, 0, 5] = 0.25
    v[0, 0, 5] *= small
    c = R.Cache(1, hkv, d, n, kv, 0, seed=1)
    (c.k, c.ks), (c.v, c.vs) = (tuple(x.repeat(B, *([1] * (x.dim() - 1))) for x in R.to_cache(y, kv)) for y in (k, v))
    c.B = B
    c.to_device(tts, hq)
    q = torch.full((1, T, hq, d), top / (0.25 * d)) + 0.001 * torch.from_numpy(g.standard_normal((1, T, hq, d)).astype(np.float32))
    q = q.bfloat16()
    out, _ = run_tree(tts, c, q.cuda().repeat(B, 1, 1, 1), [n - T] * B, [T] * B, None, T, 1.0)
    ref, mag = attend(c, q[0].double(), n - T, T, None, 1.0)
    check_tree(out, ref[None].expand(B, -1, -1, -1), mag[None].expand(B, -1, -1, -1), [T] * B)
