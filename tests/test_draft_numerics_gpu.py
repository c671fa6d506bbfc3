"""Numerics of the drafted-decoding calls at the far ends of their ranges.  References and bounds
as in test_draft_gpu.
"""
import numpy as np
import pytest
import torch

import draft_ref as R
from test_draft_gpu import check_tree, ints, masks, run_tree, tts  # noqa: F401

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


# ---------------------------------------------------------------------------
# Attention: V scales many powers of two apart
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kv", ["e4m3", "i8"])
@pytest.mark.parametrize("q_dt", ["bf16", "f32"])
@pytest.mark.parametrize("e", [20, 40, 60, 100, 118])
@pytest.mark.parametrize("T,past", [(3, 97), (20, 700), (64, 1000), (64, 0)])
def test_a_large_row_that_is_not_seen(tts, kv, q_dt, e, T, past):  # noqa: F811
    """A node's row with a V scale 2^e times the others' (finite): the nodes that do not see it
    give what they would give without it."""
    hq, hkv, d, big = 4, 2, 128, T // 2
    c = R.Cache(1, hkv, d, 1100, kv, 0, seed=3)
    c.vs[0, :, past + big] *= 2.0 ** e
    c.to_device(tts, hq)
    g = np.random.default_rng(T)
    m = masks(1, T, 3, empty=0.0)
    m[0] |= np.int64(1)
    for t in range(T):
        if t % 3:
            m[0, t] &= ~np.int64(np.uint64(1 << big).astype(np.int64))
    q = torch.from_numpy(g.standard_normal((1, T, hq, d)).astype(np.float32)).to(R.TORCH[q_dt])
    out, _ = run_tree(tts, c, q.cuda(), [past], [T], m, T, 0.1)
    ref, mag = attend(c, q[0].double(), past, T, m[0], 0.1)
    check_tree(out, ref[None], mag[None], [T])


@pytest.mark.parametrize("kv", ["e4m3", "i8"])
@pytest.mark.parametrize("q_dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 12, 30, 64])
@pytest.mark.parametrize("at", [3, 130, 700, 1180])
def test_a_large_row_of_no_weight(tts, kv, q_dt, T, at):  # noqa: F811
    """A committed row with a V scale 2^60 times the others' and a weight of 2^-90 of theirs."""
    hq, hkv, d, past = 4, 2, 128, 1190
    c = R.Cache(1, hkv, d, 1280, kv, 0, seed=4)
    k = torch.randn(1, hkv, 1280, d, generator=torch.Generator().manual_seed(T)) * 0.3
    k[0, :, at] = -2.0
    c.k, c.ks = R.to_cache(k.numpy(), kv)
    c.vs[0, :, at] *= 2.0 ** 60
    c.to_device(tts, hq)
    g = np.random.default_rng(T)
    q = torch.from_numpy(0.05 * g.standard_normal((1, T, hq, d)).astype(np.float32) + 0.25).to(R.TORCH[q_dt])
    out, _ = run_tree(tts, c, q.cuda(), [past], [T], None, T, 1.0)
    ref, mag = attend(c, q[0].double(), past, T, None, 1.0)
    check_tree(out, ref[None], mag[None], [T])


@pytest.mark.parametrize("kv", ["e4m3", "i8"])
@pytest.mark.parametrize("T", [1, 12, 30, 64])
@pytest.mark.parametrize("seed", range(4))
def test_scales_and_scores_that_both_move(tts, kv, T, seed):  # noqa: F811
    """V scales from 2^-40 to 2^40, by row or in runs, under scores that spread over 2^60: the
    largest weight, the largest weight times scale, and what was summed before all move."""
    hq, hkv, d, cap, past = 4, 2, 128, 1500, 1400
    g = np.random.default_rng(100 * T + seed)
    c = R.Cache(1, hkv, d, cap, kv, 0, seed=5 + seed)
    run = (1, 7, 64, 300)[seed]
    c.vs *= torch.from_numpy(np.exp2(np.repeat(g.integers(-40, 41, cap // run + 1), run)[:cap]).astype(np.float32))
    c.to_device(tts, hq)
    # scores of standard deviation about 6: 2^+-30 between the largest and the smallest
    q = torch.from_numpy(g.standard_normal((1, T, hq, d)).astype(np.float32)).bfloat16()
    m = masks(1, T, seed, empty=0.0)
    out, _ = run_tree(tts, c, q.cuda(), [past], [T], m, T, 6.0 * d ** -0.5)
    ref, mag = attend(c, q[0].double(), past, T, m[0], 6.0 * d ** -0.5)
    # scores of up to 40 in f32: 2^-24 of a sum of magnitudes of about 60, a few roundings, move a
    # weight by up to 2e-5 of itself; a weight whose tile's maximum moved later is rounded twice
    # (f16: 2^-11 each)
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 3e-5) * mag + 1e-5 * ref.abs().amax(-1, keepdim=True)
    assert ((out[0].cpu().double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("kv", ["e4m3", "i8"])
@pytest.mark.parametrize("q_dt", ["bf16", "f32"])
@pytest.mark.parametrize("e", [-90, -40, 40, 60])
def test_k_scales_and_queries_that_cancel(tts, kv, q_dt, e):  # noqa: F811
    """K scales times 2^e under queries times 2^-e: the scores are ordinary ones."""
    hq, hkv, d, past = 4, 2, 128, 900
    T = 11
    c = R.Cache(1, hkv, d, 1024, kv, 0, seed=8)
    c.ks *= 2.0 ** e
    c.to_device(tts, hq)
    q = torch.randn(1, T, hq, d, generator=torch.Generator().manual_seed(T)).to(R.TORCH[q_dt]) * 2.0 ** -e
    out, _ = run_tree(tts, c, q.cuda(), [past], [T], None, T, 0.1)
    ref, mag = attend(c, q[0].double(), past, T, None, 0.1)
    check_tree(out, ref[None], mag[None], [T])


# ---------------------------------------------------------------------------
# Attention: infinities in committed rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kv", ["bf16", "f32"])
@pytest.mark.parametrize("q_dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 5, 12, 30, 64])
@pytest.mark.parametrize("d,page,cap,past", [(128, 0, 512, 400), (64, 16, 768, 600), (128, 16, 4096, 3900), (64, 0, 2048, 1900)])
def test_infinities_in_committed_rows(tts, kv, q_dt, T, d, page, cap, past):  # noqa: F811
    """An infinite committed V entry gives that infinity in its column for every node, whatever the
    number of query rows; infinities of both signs, or a NaN, give NaN; other columns are exact."""
    hq, hkv, B = 4, 2, 2
    c = R.Cache(B, hkv, d, cap, kv, page, seed=6, fill=[past + T, past + T])
    inf = float("inf")
    for col, puts in ((3, [(7, inf)]), (4, [(past - 1, -inf)]), (9, [(130, inf), (131, inf)]),
                      (33, [(1, inf), (300, -inf)]), (50, [(64, float("nan"))]), (51, [(200, -inf), (201, float("nan"))])):
        for pos, x in puts:
            at, row = c.at(1, pos)
            c.v[at, :, row, col] = x
    c.to_device(tts, hq)
    q = torch.randn(B, T, hq, d, generator=torch.Generator().manual_seed(T)).to(R.TORCH[q_dt])
    out, ef = run_tree(tts, c, q.cuda(), [past] * B, [T] * B, None, T, 0.1)
    assert ef == 0
    ref, mag = (torch.stack(x) for x in zip(*(attend(c, q[b].double(), past, T, None, 0.1, b) for b in range(B))))
    check_tree(out[:1], ref[:1], mag[:1], [T])
    o = out[1].cpu().double()
    assert (o[..., 3] == inf).all() and (o[..., 4] == -inf).all() and (o[..., 9] == inf).all()
    assert o[..., 33].isnan().all() and o[..., 50].isnan().all() and o[..., 51].isnan().all()
    fine = [i for i in range(d) if i not in (3, 4, 9, 33, 50, 51)]
    check_tree(out[1:, ..., fine], ref[1:, ..., fine], mag[1:, ..., fine], [T])


# ---------------------------------------------------------------------------
# Attention: poisoned node rows where windows are cut over CTAs, page sizes of every box
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kv", ["bf16", "i8", "e4m3", "f32"])
@pytest.mark.parametrize("q_dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [10, 40])
def test_poisoned_node_rows_in_cut_windows(tts, kv, q_dt, T):  # noqa: F811
    """A capacity above what one CTA takes whole: noted V rows and scores that are all NaN pass
    through partial rows and their merge; an empty mask over no committed rows gives 0."""
    hq, hkv, d, cap, past = 4, 2, 128, 4096, [0, 1500, 3001]
    B, bad_v, bad_k = 3, 3, 1
    g = np.random.default_rng(T)
    c = R.Cache(B, hkv, d, cap, kv, 0, seed=7, fill=[p + T for p in past])
    m = masks(B, T, 4, empty=0.0)
    m[:, 4] = 0
    m[:, 6] = 1 << bad_k                        # with no committed rows: nothing but a NaN score
    m[:, 8] |= (1 << bad_v) | (1 << bad_k)
    for b, p in enumerate(past):
        if kv in R.TOP:
            c.vs[b, :, p + bad_v] = float("inf")
            c.ks[b, :, p + bad_k] = float("nan")
        else:
            c.v[b, :, p + bad_v, 5] = float("inf")
            c.v[b, :, p + bad_v, 6] = float("nan")
            c.k[b, :, p + bad_k, 0] = float("nan")
    c.to_device(tts, hq)
    q = torch.from_numpy(g.standard_normal((B, T, hq, d)).astype(np.float32)).to(R.TORCH[q_dt])
    out, ef = run_tree(tts, c, q.cuda(), past, [T] * B, m, T, 0.1)
    assert ef == 0
    ref, mag = R.tree_attn(c, q.double(), past, [T] * B, m, 0.1)
    o = out.cpu().double()
    for b in range(B):
        for t in range(T):
            got, want = out[b:b + 1, t:t + 1], (ref[b:b + 1, t:t + 1], mag[b:b + 1, t:t + 1])
            if m[b, t] >> bad_k & 1:
                assert o[b, t].isnan().all(), (b, t)
            elif m[b, t] >> bad_v & 1:
                if kv in R.TOP:
                    assert not o[b, t].isfinite().any(), (b, t)
                else:
                    assert (o[b, t, :, 5] == float("inf")).all() and o[b, t, :, 6].isnan().all(), (b, t)
                    fine = [i for i in range(d) if i not in (5, 6)]
                    check_tree(got[..., fine], *(x[..., fine] for x in want), [1])
            else:
                check_tree(got, *want, [1])
    assert (o[0, 4] == 0).all()


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("page", [2, 8, 32, 128, 256])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [512, 2048])
def test_pages_of_every_size(tts, kv, page, d, cap):  # noqa: F811
    hq, hkv, B, T = 4, 2, 3, 9
    past = [cap - T, 3, cap // 2 - 5]
    c = R.Cache(B, hkv, d, cap, kv, page, seed=page, fill=[p + T for p in past]).to_device(tts, hq)
    q = torch.randn(B, T, hq, d, generator=torch.Generator().manual_seed(page)).bfloat16()
    m = masks(B, T, page)
    out, ef = run_tree(tts, c, q.cuda(), past, [T] * B, m, T, d ** -0.5)
    assert ef == 0
    ref, mag = (torch.stack(x) for x in zip(*(attend(c, q[b].double(), past[b], T, m[b], d ** -0.5, b) for b in range(B))))
    none = torch.tensor([[not (past[b] or int(m[b, t]) & ((1 << T) - 1)) for t in range(T)] for b in range(B)])
    ref[none], mag[none] = 0.0, 0.0
    check_tree(out, ref, mag, [T] * B)
