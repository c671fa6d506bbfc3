"""The drafted-decoding calls against 64-bit restatements (draft_ref): rotary rows and scaled
tables, rows quantised into a cache and read back, attention of drafted trees over f32, bf16
and 8-bit caches, and the commit of an accepted path -- alone and as they are used together.

Tolerances, fixed before the first run:
* rotary rows in f32: 2e-6 of the row's largest magnitude, the norm-and-rotation bound of the
  other tests (about 20 roundings of 2^-24); bf16 adds half a step, 2^-8 of the value.
* tables: half a step of f32 (2^-24 of the entry) plus 1e-9 for the angle.
* 8-bit codes and scales: the same bits; f32 read-back: the same bits.
* attention with f32 q: 1e-5 of the row's largest magnitude (the f32 bound of the other
  attention tests), plus 1e-5 of the weighted mean |v| where outputs cancel.
* attention with bf16 q: the output's half step (2^-8 of it), and the weights' half step,
  which moves the output by at most 2^-8 of the weighted mean |v|; plus the f32 terms.
"""
import math

import numpy as np
import pytest
import torch

import draft_ref as R
from gpu_helpers import bits

pytestmark = pytest.mark.gpu

I32 = torch.int32


@pytest.fixture(scope="module")
def tts(cuda_dev):
    from autoregressive_codebook_tts_gb300 import build
    build.build()
    from autoregressive_codebook_tts_gb300 import tts as mod
    return mod


def flag():
    return torch.zeros(1, dtype=I32, device="cuda")


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


# ---------------------------------------------------------------------------
# Rotary rows and tables
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("max_pos,rot,kind,factor", [
    (1, 2, "none", 1.0), (33, 128, "none", 1.0), (1025, 6, "linear", 4.0), (300, 30, "base", 3.0),
    (4096, 128, "parts", 8.0), (20000, 64, "parts", 2.5), (2048, 4, "base", 16.0)])
def test_scaled_tables(tts, max_pos, rot, kind, factor):
    kw = dict(kind=kind, factor=factor)
    ref = R.table(max_pos, rot, 5e5, L=1024, low=1.0, high=32.0, attn=1.1, **kw)
    cs = torch.full((max_pos + 1, rot // 2, 2), float("nan"), device="cuda")
    tts.tts_rope_table_scaled(cs[:max_pos], max_pos, rot, 5e5, original_max_pos=1024, attn_scale=1.1, **kw)
    got = cs.cpu().double().numpy()
    assert np.isnan(got[max_pos]).all()
    assert (np.abs(got[:max_pos] - ref) <= 2.0 ** -24 * np.abs(ref) + 1e-9).all()


def test_unscaled_table_is_the_earlier_one(tts):
    a, b = torch.empty(4096, 64, 2, device="cuda"), torch.empty(4096, 64, 2, device="cuda")
    tts.tts_rope_table(a, 4096, 128, 1e6)
    tts.tts_rope_table_scaled(b, 4096, 128, 1e6)
    assert (a - b).abs().max().item() <= 2.0 ** -24 + 1e-9


@pytest.mark.parametrize("rows,hq,hkv,d,rot,inter,norm,dt,odt", [
    (1, 16, 8, 128, 128, False, True, "f32", "f32"),
    (5, 3, 1, 128, 128, True, True, "f32", "bf16"),
    (7, 4, 4, 64, 64, False, False, "bf16", "f32"),
    (3, 2, 1, 64, 22, False, True, "f32", "f32"),       # half of 11: partners not vector-aligned
    (3, 2, 1, 128, 2, True, False, "f32", "f32"),
    (4, 5, 3, 128, 126, True, True, "bf16", "bf16"),
    (2, 1, 1, 64, 2, False, True, "f32", "f32"),
    (700, 16, 8, 128, 32, False, True, "f32", "bf16"),  # four heads a warp
    (900, 15, 4, 64, 48, True, False, "bf16", "bf16"),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_rows(tts, rows, hq, hkv, d, rot, inter, norm, dt, odt, in_place):
    if in_place and dt != odt:
        pytest.skip("in place has one type")
    g = torch.Generator().manual_seed(rows * 7 + rot)
    width = (hq + 2 * hkv) * d + 8
    x = torch.randn(rows, width, generator=g).to(R.TORCH[dt])
    pos = torch.randint(0, 200, (rows,), generator=g, dtype=I32)
    cs = torch.from_numpy(R.table(200, rot, 1e4)).float().contiguous()
    gq, gk = torch.rand(d, generator=g) + 0.5, torch.rand(d, generator=g) + 0.5
    dx = x.cuda()
    q, k = dx[:, :hq * d], dx[:, hq * d:(hq + hkv) * d]
    if in_place:
        qo, ko = q, k
    else:
        qo = torch.full((rows, hq * d + 16), float("nan"), dtype=R.TORCH[odt], device="cuda")[:, :hq * d]
        ko = torch.full((rows, hkv * d), float("nan"), dtype=R.TORCH[odt], device="cuda")
    ef = flag()
    tts.tts_rope_rows(q, k, qo, ko, pos.cuda(), hq, hkv, d, cs.cuda(), gamma_q=gq.cuda() if norm else None,
                      gamma_k=gk.cuda() if norm else None, interleaved=inter, err_flag=ef)
    assert ef.item() == 0
    xd = x.double()
    for got, h0, h, gam in ((qo, 0, hq, gq), (ko, hq, hkv, gk)):
        ref = R.rope(xd[:, h0 * d:(h0 + h) * d].reshape(rows, h, d), pos, cs, rot, inter, gam if norm else None)
        got = got.cpu().double().reshape(rows, h, d)
        bound = 2e-6 * ref.abs().amax(-1, keepdim=True) + (2.0 ** -8 * ref.abs() if odt == "bf16" else 0)
        assert ((got - ref).abs() <= bound).all()
    if in_place:   # the v columns and the padding are untouched
        assert torch.equal(dx[:, (hq + hkv) * d:].cpu(), x[:, (hq + hkv) * d:])
    else:
        assert torch.equal(dx.cpu(), x)


def test_rope_rows_without_k_and_bad_positions(tts):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(4, 128, generator=g)
    cs = torch.from_numpy(R.table(10, 64, 1e4)).float().contiguous()
    pos = torch.tensor([-3, 9, 10, 0], dtype=I32)
    out, ef = torch.empty(4, 128, device="cuda"), flag()
    tts.tts_rope_rows(x.cuda(), None, out, None, pos.cuda(), 2, 0, 64, cs.cuda(), err_flag=ef)
    assert ef.item() == tts.EFLAG_POS_RANGE
    ref = R.rope(x.double().reshape(4, 2, 64), pos.clamp(0, 9), cs, 64, False)
    assert ((out.cpu().double().reshape(4, 2, 64) - ref).abs() <= 2e-6 * ref.abs().amax()).all()
    # position 0 of an unnormed row is the row itself
    assert torch.equal(out[3].cpu(), x[3])


def test_rope_rows_agree_with_the_norm_rope_call(tts):
    g = torch.Generator().manual_seed(2)
    q, k = torch.randn(6, 2048, generator=g).cuda(), torch.randn(6, 1024, generator=g).cuda()
    gq, gk = torch.rand(128, generator=g).cuda(), torch.rand(128, generator=g).cuda()
    pos = ints([0, 5, 100, 255, 17, 1])
    cs = torch.empty(256, 64, 2, device="cuda")
    tts.tts_rope_table(cs, 256, 128, 1e6)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    tts.tts_rope_rows(q, k, qo, ko, pos, 16, 8, 128, cs, gamma_q=gq, gamma_k=gk)
    tts.tts_qk_norm_rope(q, k, gq, gk, pos, 16, 8, 128, 1e-6, cs, 256)
    assert (qo - q).abs().max() <= 4e-6 * q.abs().max() and (ko - k).abs().max() <= 4e-6 * k.abs().max()


# ---------------------------------------------------------------------------
# Cache rows
# ---------------------------------------------------------------------------
def border_rows(n, hkv, d, seed):
    """Rows that hold values on and next to borders between codes, tiny and huge rows, zero
    rows and rows with a NaN or an infinity."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((n, hkv, d)).astype(np.float32) * np.exp(g.standard_normal((n, hkv, 1)) * 3).astype(np.float32)
    flat = x.reshape(-1, d)
    for i in range(0, len(flat), 5):
        # quotients k + 1/2 (int8) and halves between 4-bit floats, give or take a last place
        s = np.float32(2.0) ** g.integers(-20, 20)
        top = np.float32(127.0 if i % 2 else 448.0)
        near = g.integers(-120, 120, d) + 0.5 if i % 2 else R.nearest_code(g.uniform(0, 400, d), "e4m3") * (1 + 1 / 16)
        y = (near * s).astype(np.float32)
        y = np.nextafter(y, np.float32(g.choice([-np.inf, np.inf])), dtype=np.float32) if i % 3 else y
        y[0] = top * s
        flat[i] = y * g.choice([np.float32(1), np.float32(1.37)])
    flat[1] = 0
    flat[2, 3] = np.nan
    flat[3, 5] = np.inf
    flat[4, 0] = -np.inf
    flat[6] = (g.integers(-3, 4, d) * 2.0 ** -149).astype(np.float32)
    flat[7] = (g.standard_normal(d) * 2.0 ** -130).astype(np.float32)
    flat[8] = (g.standard_normal(d) * 1e37).astype(np.float32)
    flat[9, 1:] = 0
    return x


@pytest.mark.parametrize("kv", ["i8", "e4m3", "bf16", "f32"])
@pytest.mark.parametrize("src", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,hkv,d,cap,page", [(3, 1, 8, 128, 40, 0), (2, 19, 3, 64, 64, 16), (1, 300, 2, 128, 304, 0),
                                                (2, 700, 8, 64, 1024, 1)])
def test_rows_written_and_read_back(tts, kv, src, B, T, hkv, d, cap, page):
    c = R.Cache(B, hkv, d, cap, kv, page, seed=T).to_device(tts, 2 * hkv)
    k = torch.from_numpy(border_rows(B * T, hkv, d, 1)).to(R.TORCH[src])
    v = torch.from_numpy(border_rows(B * T, hkv, d, 2)).to(R.TORCH[src])
    start = [min(cap - T, 3 * b + 1) for b in range(B)]
    count = [T if b != 1 else T // 2 for b in range(B)]
    rows = torch.cat([k.flatten(1), v.flatten(1), torch.zeros(B * T, 8, dtype=k.dtype)], 1).cuda()
    kd = hkv * d
    ef = flag()
    tts.tts_kv_write_rows(rows[:, :kd], rows[:, kd:2 * kd], c.cache, c.desc, ints(start), T, n_rows=ints(count), err_flag=ef)
    ko = torch.full((B * T, kd), 7.0, device="cuda")
    vo = torch.full((B * T, kd), 7.0, device="cuda")
    kb, vb = ko.bfloat16(), vo.bfloat16()
    tts.tts_kv_read_rows(c.cache, c.desc, ints(start), T, ko, vo, n_rows=ints(count), err_flag=ef)
    tts.tts_kv_read_rows(c.cache, c.desc, ints(start), T, kb, vb, n_rows=ints(count), err_flag=ef)
    assert ef.item() == 0
    # the definition, on the host copy
    for x, t, s, out, outb in ((k, c.k, c.ks, ko, kb), (v, c.v, c.vs, vo, vb)):
        code, scale = R.to_cache(x.float().numpy(), kv)
        out, outb = out.cpu().reshape(B, T, hkv, d), outb.cpu().reshape(B, T, hkv, d)
        for b in range(B):
            for i in range(T):
                if i >= count[b]:
                    assert (out[b, i] == 7).all() and (outb[b, i] == 7).all()
                    continue
                at, row = c.at(b, start[b] + i)
                t[at, :, row] = code[b * T + i]
                want = code[b * T + i].float()
                if s is not None:
                    s[at, :, row] = scale[b * T + i]
                    want = want * scale[b * T + i][:, None]
                assert np.array_equal(bits((out[b, i] + 0).numpy()), bits((want + 0).numpy())) or (
                    torch.equal(out[b, i].nan_to_num(1e30), want.nan_to_num(1e30)))
                assert torch.equal(outb[b, i].float().nan_to_num(1e30), want.bfloat16().float().nan_to_num(1e30))
    # every byte of the cache: the rows written, and all the others as they were (zeros may
    # differ in sign of their code, NaN scales in their payload)
    for got, ref in ((c.dk, c.k), (c.dv, c.v), (c.dks, c.ks), (c.dvs, c.vs)):
        if ref is not None:
            a, b = got.cpu().float(), ref.float()
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0), b.nan_to_num(0))


# Every border of a format, both signs, in rows whose largest magnitude is Q 2^e: the scale is then
# 2^e exactly (Q * f32(1 / Q) = 1 for both Q), the quotients are the borders exactly, and each has
# two nearest codes, of which the even one is to be taken.  All entries fit in bf16.
@pytest.mark.parametrize("kv", ["i8", "e4m3"])
@pytest.mark.parametrize("src", ["f32", "bf16"])
def test_ties_take_the_even_code(tts, kv, src):
    if kv == "i8":
        codes = np.arange(-127, 128)
        borders = codes[:-1] + 0.5
        want = np.where(codes[:-1] % 2 == 0, codes[:-1], codes[:-1] + 1) & 0xff
    else:
        value = lambda c: (c % 8) * 2.0 ** -9 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 10)  # noqa: E731
        low = np.arange(126)
        mid = np.array([(value(c) + value(c + 1)) / 2 for c in low])
        even = np.where(low % 2 == 0, low, low + 1)
        borders, want = np.concatenate([mid, -mid]), np.concatenate([even, even | 0x80])
    top, n = (127.0 if kv == "i8" else 448.0), len(borders)
    quot, code = np.zeros((2, 128)), np.zeros((2, 128), np.int64)
    for i in range(2):
        part = slice(i * (n // 2), (i + 1) * (n // 2))
        quot[i, 0], code[i, 0] = top, 127 if kv == "i8" else 126
        quot[i, 1:1 + n // 2], code[i, 1:1 + n // 2] = borders[part], want[part]
    exps = list(range(-30, 31))
    x64 = np.stack([quot * 2.0 ** e for e in exps])                     # [61][2][128]
    x = torch.from_numpy(x64.astype(np.float32)).to(R.TORCH[src])
    assert np.array_equal(x.double().numpy(), x64)
    rows = x.reshape(len(exps), 256).cuda()                             # two kv heads a row
    c = R.Cache(1, 2, 128, 64, kv, 0, seed=5).to_device(tts, 4)
    tts.tts_kv_write_rows(rows, rows, c.cache, c.desc, ints([0]), len(exps))
    for t, scale in ((c.dk, c.dks), (c.dv, c.dvs)):
        got = t.view(torch.uint8)[0, :, :len(exps)].permute(1, 0, 2).cpu().numpy().astype(np.int64)
        zero = (code & 0x7f) == 0 if kv == "e4m3" else np.zeros_like(code, bool)
        got = np.where(zero[None] & (got == 0x80), 0, got)              # (a zero's sign)
        ref = np.where(zero, 0, code)
        assert np.array_equal(got, np.broadcast_to(ref, got.shape))
        assert np.array_equal(scale[0, :, :len(exps)].cpu().double().numpy(),
                              np.broadcast_to(2.0 ** np.array(exps), (2, len(exps))))


def test_rows_out_of_range_are_skipped_and_flagged(tts):
    for page in (0, 16):
        c = R.Cache(4, 2, 64, 64, "i8", page, seed=5).to_device(tts, 4)
        x = torch.randn(4 * 3, 128, generator=torch.Generator().manual_seed(3)).cuda()
        ef = flag()
        tts.tts_kv_write_rows(x, x, c.cache, c.desc, ints([-2, 62, 2 ** 31 - 1, -2 ** 31]), 3, err_flag=ef)
        assert ef.item() == tts.EFLAG_POS_RANGE
        code, scale = R.to_cache(x.cpu().reshape(12, 2, 64).numpy(), "i8")
        for b, i, pos in ((0, 2, 0), (1, 0, 62), (1, 1, 63)):
            at, row = c.at(b, pos)
            for t, s in ((c.k, c.ks), (c.v, c.vs)):
                t[at, :, row], s[at, :, row] = code[b * 3 + i], scale[b * 3 + i]
        assert all(torch.equal(a, b) for a, b in zip(c.back(), c.host()))
        out = torch.full((12, 128), 5.0, device="cuda")
        ef = flag()
        tts.tts_kv_read_rows(c.cache, c.desc, ints([-2, 62, 2 ** 31 - 1, -2 ** 31]), 3, out, out.clone(), err_flag=ef)
        assert ef.item() == tts.EFLAG_POS_RANGE
        untouched = [0, 1, 5, 6, 7, 8, 9, 10, 11]
        assert (out[untouched] == 5).all() and (out[[2, 3, 4]] != 5).any(1).all()
        ef = flag()
        tts.tts_kv_write_rows(x, x, c.cache, c.desc, ints([0, 0, 0, 0]), 3, n_rows=ints([0, -1, 0, 0]), err_flag=ef)
        assert ef.item() == tts.EFLAG_NVALID
        assert all(torch.equal(a, b) for a, b in zip(c.back(), c.host()))
    # a page id outside the pool
    c = R.Cache(2, 2, 64, 64, "e4m3", 16, seed=6)
    c.bt[1, 2] = -1
    c.to_device(tts, 4)
    x, ef = torch.randn(2 * 20, 128).cuda(), flag()
    before = c.back()
    tts.tts_kv_write_rows(x, x, c.cache, c.desc, ints([0, 44]), 20, n_rows=ints([0, 20]), err_flag=ef)
    assert ef.item() == tts.EFLAG_PAGE
    after = c.back()
    page = int(c.bt[1, 3])
    for a, b in zip(before, after):
        changed = (a != b).flatten(1).any(1)
        assert changed[page] and changed.sum() == 1


def test_offsets_beyond_32_bits(tts):
    # a pool of over 2^32 bytes and 2^32 entries a tensor; the streams' pages lie at its end
    hkv, d, page = 8, 128, 256
    n_pages = 2 ** 32 // (hkv * d * page) + 9
    k = torch.zeros(n_pages, hkv, page, d, dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    ks, vs = (torch.zeros(n_pages, hkv, page, device="cuda") for _ in range(2))
    bt = ints([[n_pages - 1, n_pages - 3]])
    desc = tts.kv_desc(1, 16, hkv, d, 512, "i8", paged=True, page_size=page, n_pages=n_pages, block_table=bt)
    cache = tts.kv_cache(k, v, ks, vs)
    T = 64
    g = torch.Generator().manual_seed(4)
    x, y = torch.randn(T, hkv * d, generator=g), torch.randn(T, hkv * d, generator=g)
    start = 256 - 20
    tts.tts_kv_write_rows(x.cuda(), y.cuda(), cache, desc, ints([start]), T)
    ko, vo = torch.empty(T, hkv * d, device="cuda"), torch.empty(T, hkv * d, device="cuda")
    tts.tts_kv_read_rows(cache, desc, ints([start]), T, ko, vo)
    for a, b in ((x, ko), (y, vo)):
        code, s = R.quantise(a.reshape(T, hkv, d).numpy(), "i8")
        assert np.array_equal(b.cpu().numpy().reshape(T, hkv, d), (code * s[..., None].astype(np.float64)).astype(np.float32))
    # attention reads the same rows (rows below are code 0, scale 0: scores 0, values 0)
    for q_dt in (torch.float32, torch.bfloat16):
        q = torch.randn(1, 2048, generator=g).to(q_dt).cuda()
        out = torch.empty_like(q)
        tts.tts_tree_attn(q, cache, desc, ints([start + T - 1]), 1, 0.1, out, tts.tree_workspace(desc, 1, q_dt))
        K = torch.cat([torch.zeros(start, hkv, d), ko.cpu().reshape(T, hkv, d)]).double().repeat_interleave(2, 1)
        V = torch.cat([torch.zeros(start, hkv, d), vo.cpu().reshape(T, hkv, d)]).double().repeat_interleave(2, 1)
        w = torch.softmax(torch.einsum("hd,nhd->hn", q.cpu().double().reshape(16, d), K) * 0.1, -1)
        ref = torch.einsum("hn,nhd->hd", w, V)
        mag = torch.einsum("hn,nhd->hd", w, V.abs())
        check_tree(out.reshape(1, 1, 16, d), ref[None, None], mag[None, None], [1])
    # the accepted rows move across the page border
    path = ints([[0, 30, 63]])
    tts.tts_tree_commit(cache, desc, ints([start]), torch.cat([path, path.new_zeros(1, 61)], 1), ints([3]), 64)
    tts.tts_kv_read_rows(cache, desc, ints([start]), 3, ko[:3], vo[:3])
    code, s = R.quantise(x.reshape(T, hkv, d)[[0, 30, 63]].numpy(), "i8")
    assert np.array_equal(ko[:3].cpu().numpy().reshape(3, hkv, d), (code * s[..., None].astype(np.float64)).astype(np.float32))


# ---------------------------------------------------------------------------
# Tree attention
# ---------------------------------------------------------------------------
def check_tree(out, ref, mag, nodes):
    out_d = out.cpu().double()
    bf = out.dtype == torch.bfloat16
    for b, n in enumerate(nodes):
        o, r, m = out_d[b, :n], ref[b, :n], mag[b, :n]
        bound = 1e-5 * r.abs().amax(-1, keepdim=True) + 1e-5 * m
        if bf:
            bound = bound + 2.0 ** -8 * r.abs() + 2.0 ** -8 * m
        err = (o - r).abs()
        assert (err <= bound).all(), (b, float((err - bound).max()), float(err.max()))


def run_tree(tts, c, q, past, nodes, mask, T, scale, n_nodes=True, ws=None):
    """(out [B, T, Hq, D], flag) with the output preset to 9."""
    B, _, Hq, D = q.shape
    out = torch.full_like(q, 9.0)
    ef = flag()
    ws = tts.tree_workspace(c.desc, T, q.dtype) if ws is None else ws
    tts.tts_tree_attn(q.reshape(B * T, Hq * D), c.cache, c.desc, ints(past), T, scale, out, ws,
                      n_nodes=ints(nodes) if n_nodes else None,
                      tree_mask=None if mask is None else torch.from_numpy(np.ascontiguousarray(mask)).cuda(), err_flag=ef)
    return out, ef.item()


def masks(B, T, seed, empty=0.15):
    rng = np.random.default_rng(seed)
    return np.stack([R.random_tree(T, rng, empty) for _ in range(B)])


CASES = [
    # B, T, hq, hkv, d, cap, page, past (per stream)
    (1, 1, 2, 1, 128, 8, 0, [0]),
    (2, 1, 16, 8, 128, 300, 0, [299, 0]),
    (3, 5, 8, 8, 64, 200, 0, [0, 63, 64]),
    (2, 7, 8, 2, 128, 512, 16, [129, 505]),
    (2, 64, 4, 2, 128, 448, 64, [0, 320]),
    (1, 64, 8, 2, 64, 700, 4, [636]),
    (4, 16, 6, 3, 128, 1100, 0, [1, 127, 128, 1084]),
    (2, 33, 2, 2, 128, 640, 1, [95, 607]),
    (1, 20, 4, 4, 64, 1300, 4, [1280]),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("kv", ["f32", "bf16", "i8", "e4m3"])
@pytest.mark.parametrize("q_dt", ["f32", "bf16"])
def test_tree_attention(tts, case, kv, q_dt):
    B, T, hq, hkv, d, cap, page, past = CASES[case]
    rng = np.random.default_rng(case)
    nodes = [T if b % 2 == 0 else max(1, T - 3) for b in range(B)]
    c = R.Cache(B, hkv, d, cap, kv, page, seed=case, fill=[p + n for p, n in zip(past, nodes)]).to_device(tts, hq)
    q = torch.from_numpy(rng.standard_normal((B, T, hq, d)).astype(np.float32)).to(R.TORCH[q_dt])
    m = masks(B, T, case)
    scale = d ** -0.5
    out, ef = run_tree(tts, c, q.cuda(), past, nodes, m, T, scale)
    assert ef == 0
    ref, mag = R.tree_attn(c, q.double(), past, nodes, m, scale)
    check_tree(out, ref, mag, nodes)
    for b in range(B):
        assert (out[b, nodes[b]:] == 9).all()
    # the chain, all T nodes where they fit
    if all(p + T <= cap for p in past) and kv in ("f32", "i8"):
        full = [T] * B
        c = R.Cache(B, hkv, d, cap, kv, page, seed=case + 50, fill=[p + T for p in past]).to_device(tts, hq)
        out, ef = run_tree(tts, c, q.cuda(), past, full, None, T, scale, n_nodes=False)
        assert ef == 0
        check_tree(out, *R.tree_attn(c, q.double(), past, full, None, scale), full)


@pytest.mark.parametrize("kv", ["bf16", "i8", "e4m3", "f32"])
@pytest.mark.parametrize("q_dt", ["bf16", "f32"])
@pytest.mark.parametrize("page", [0, 16])
def test_tree_attention_over_long_ragged_windows(tts, kv, q_dt, page):
    # more work than one wave of CTAs: items of many tiles cut across CTAs, and whole ones
    B, T, hq, hkv, d, cap = 5, 12, 4, 2, 128, 4096
    past = [4084, 1, 2500, 700, 3333]
    rng = np.random.default_rng(9)
    c = R.Cache(B, hkv, d, cap, kv, page, seed=3, fill=[p + T for p in past]).to_device(tts, hq)
    q = torch.from_numpy(rng.standard_normal((B, T, hq, d)).astype(np.float32) * 2).to(R.TORCH[q_dt])
    m = masks(B, T, 5)
    out, ef = run_tree(tts, c, q.cuda(), past, [T] * B, m, T, d ** -0.5)
    assert ef == 0
    check_tree(out, *R.tree_attn(c, q.double(), past, [T] * B, m, d ** -0.5), [T] * B)
    # again with the same workspace, and with another's leftovers in it: the same bytes
    ws = tts.tree_workspace(c.desc, T, R.TORCH[q_dt])
    ws.fill_(0xFF)
    again, _ = run_tree(tts, c, q.cuda(), past, [T] * B, m, T, d ** -0.5, ws=ws)
    assert torch.equal(out, again)


def test_single_token_form_agrees_with_decode_attention(tts):
    B, hq, hkv, d, cap = 6, 16, 8, 128, 2048
    g = torch.Generator().manual_seed(8)
    k, v = (torch.randn(B, hkv, cap, d, generator=g).cuda() for _ in range(2))
    q = torch.randn(B, hq * d, generator=g).cuda()
    past = ints([0, 1, 200, 1023, 1500, 2047])
    desc = tts.kv_desc(B, hq, hkv, d, cap, "f32")
    a, b = torch.empty(B, hq, d, device="cuda"), torch.empty(B, hq, d, device="cuda")
    tts.tts_decode_attn(q, k, v, desc, past + 1, d ** -0.5, a, tts.workspace(desc))
    tts.tts_tree_attn(q, tts.kv_cache(k, v), desc, past, 1, d ** -0.5, b, tts.tree_workspace(desc, 1))
    assert (a - b).abs().max() <= 2e-5 * a.abs().max()


def test_tree_attention_on_strided_queries(tts):
    B, T, hq, hkv, d, cap = 2, 9, 4, 2, 128, 200
    c = R.Cache(B, hkv, d, cap, "i8", 0, seed=1, fill=[150, 150]).to_device(tts, hq)
    for dt in (torch.float32, torch.bfloat16):
        x = torch.randn(B * T, (hq + 2 * hkv) * d + 8, generator=torch.Generator().manual_seed(2)).to(dt).cuda()
        q = x[:, :hq * d]
        out, ef = torch.empty(B, T, hq, d, dtype=dt, device="cuda"), flag()
        tts.tts_tree_attn(q, c.cache, c.desc, ints([141, 100]), T, 0.09, out, tts.tree_workspace(c.desc, T, dt), err_flag=ef)
        assert ef.item() == 0
        ref = R.tree_attn(c, q.cpu().double().reshape(B, T, hq, d), [141, 100], [T, T], None, 0.09)
        check_tree(out, *ref, [T, T])


@pytest.mark.parametrize("q_dt", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.09, 30.0])
def test_tree_attention_scales(tts, q_dt, scale):
    # equal weights, reversed order, one-hot weights (differences far below the smallest 2^x)
    B, T, hq, hkv, d = 1, 6, 4, 2, 128
    c = R.Cache(B, hkv, d, 700, "bf16", 0, seed=4, fill=[650]).to_device(tts, hq)
    q = torch.randn(B, T, hq, d, generator=torch.Generator().manual_seed(3)).to(R.TORCH[q_dt])
    m = masks(B, T, 2)
    out, _ = run_tree(tts, c, q.cuda(), [644], [T], m, T, scale)
    if scale == 30.0 and q_dt == "f32":
        # scores near 1000: their f32 rounding (2^-24 of the sum of magnitudes, times 30)
        # moves a weight by up to 1e-3 of itself
        ref, mag = R.tree_attn(c, q.double(), [644], [T], m, scale)
        assert ((out.cpu().double() - ref).abs() <= 2e-3 * mag + 1e-5).all()
    elif scale == 30.0:
        ref, mag = R.tree_attn(c, q.double(), [644], [T], m, scale)
        assert ((out.cpu().double() - ref).abs() <= (2e-3 + 2.0 ** -7) * mag + 1e-5).all()
    else:
        check_tree(out, *R.tree_attn(c, q.double(), [644], [T], m, scale), [T])


@pytest.mark.parametrize("kv", ["f32", "bf16", "i8", "e4m3"])
@pytest.mark.parametrize("q_dt", ["f32", "bf16"])
@pytest.mark.parametrize("past", [0, 60, 500])
def test_nothing_masked_reaches_the_result(tts, kv, q_dt, past):
    """Node rows that hold NaN or infinity: the nodes that do not see them are exact, those
    that see them are not finite where the formula is not; an empty mask gives 0."""
    T, hq, hkv, d, cap = 10, 4, 2, 128, 700
    rng = np.random.default_rng(3)
    c = R.Cache(1, hkv, d, cap, kv, 0, seed=6, fill=[past + T])
    m = np.array([[1, 2, 4 | 1, 8, 0, 32 | 2, 64 | 8, 128, 256 | 4, -2 ** 63 | 512]], np.int64)  # bits past T are ignored
    bad_v, bad_k = 3, 1        # nodes whose rows are poisoned
    if kv in R.TOP:
        c.vs[0, :, past + bad_v] = float("inf")
        c.ks[0, :, past + bad_k] = float("nan")
    else:
        c.v[0, :, past + bad_v, 5] = float("inf")
        c.v[0, :, past + bad_v, 6] = float("nan")
        c.k[0, :, past + bad_k, 0] = float("nan")
    c.to_device(tts, hq)
    q = torch.from_numpy(rng.standard_normal((1, T, hq, d)).astype(np.float32)).to(R.TORCH[q_dt])
    out, ef = run_tree(tts, c, q.cuda(), [past], [T], m, T, 0.1)
    assert ef == 0
    ref, mag = R.tree_attn(c, q.double(), [past], [T], m, 0.1)
    o = out.cpu().double()
    for t in range(T):
        if m[0, t] >> bad_k & 1:
            assert o[0, t].isnan().all(), t
        elif m[0, t] >> bad_v & 1:
            if kv in R.TOP:
                assert not o[0, t][c_nonzero(c, past + bad_v, hq)].isfinite().any(), t
            else:
                assert o[0, t, :, 5].isinf().all() and o[0, t, :, 6].isnan().all(), t
                fine = [i for i in range(d) if i not in (5, 6)]
                check_tree(out[:, t:t + 1, :, fine], ref[:, t:t + 1, :, fine], mag[:, t:t + 1, :, fine], [1])
        else:
            check_tree(out[:, t:t + 1], ref[:, t:t + 1], mag[:, t:t + 1], [1])
    if past == 0:
        assert (o[0, 4] == 0).all()


def c_nonzero(c, pos, hq):
    """Entries of the query heads whose V code at pos is not 0 (0 * infinity is NaN too)."""
    return torch.ones(hq, c.d, dtype=torch.bool)


def test_windows_out_of_range_are_clamped_and_flagged(tts):
    T, hq, hkv, d, cap = 4, 4, 2, 128, 300
    q = torch.randn(1, T, hq, d, generator=torch.Generator().manual_seed(1))
    c = R.Cache(1, hkv, d, cap, "bf16", 0, seed=2).to_device(tts, hq)
    for q_dt in ("f32", "bf16"):
        qq = q.to(R.TORCH[q_dt])
        for past, nodes, p2, n2 in ((-5, 4, 0, 4), (298, 4, 298, 2), (300, 4, 300, 0), (400, 2, 300, 0), (10, 9, 10, 4),
                                    (10, -1, 10, 0), (2 ** 31 - 1, 4, 300, 0), (-2 ** 31, 1, 0, 1)):
            out, ef = run_tree(tts, c, qq.cuda(), [past], [nodes], None, T, 0.1)
            assert ef == tts.EFLAG_NVALID, (past, nodes)
            check_tree(out, *R.tree_attn(c, qq.double(), [p2], [n2], None, 0.1), [n2])
            assert (out[0, n2:] == 9).all()
        out, ef = run_tree(tts, c, qq.cuda(), [100], [0], None, T, 0.1)
        assert ef == 0 and (out == 9).all()


def test_page_ids(tts):
    T, hq, hkv, d, cap = 3, 4, 2, 64, 640
    c = R.Cache(2, hkv, d, cap, "i8", 16, seed=2)
    c.bt[0, 7] = c.n_pages           # in stream 0's window: reads page 0
    c.bt[1, 20:] = -1                # past stream 1's window: never read
    c.to_device(tts, hq)
    q = torch.randn(2, T, hq, d, generator=torch.Generator().manual_seed(1))
    c.bt[0, 7] = 0
    for q_dt in ("f32", "bf16"):
        qq = q.to(R.TORCH[q_dt])
        out, ef = run_tree(tts, c, qq.cuda(), [500, 317], [T, T], None, T, 0.1)
        assert ef == tts.EFLAG_PAGE
        check_tree(out, *R.tree_attn(c, qq.double(), [500, 317], [T, T], None, 0.1), [T, T])
        out, ef = run_tree(tts, c, qq.cuda(), [100, 317], [T, T], None, T, 0.1)
        assert ef == 0


@pytest.mark.parametrize("q_dt", ["f32", "bf16"])
def test_many_streams(tts, q_dt):
    # more streams than lanes of the walk's scan, many items a CTA, some streams empty
    B, T, hq, hkv, d, cap = 150, 2, 2, 1, 64, 512
    past = [(b * 37) % 500 for b in range(B)]
    nodes = [(b % 3) for b in range(B)]
    c = R.Cache(B, hkv, d, cap, "bf16", 0, seed=1).to_device(tts, hq)
    q = torch.randn(B, T, hq, d, generator=torch.Generator().manual_seed(1)).to(R.TORCH[q_dt])
    out, ef = run_tree(tts, c, q.cuda(), past, nodes, None, T, 0.1)
    assert ef == 0
    check_tree(out, *R.tree_attn(c, q.double(), past, nodes, None, 0.1), nodes)
    for b in range(B):
        assert (out[b, nodes[b]:] == 9).all()


@pytest.mark.parametrize("kv", ["bf16", "i8", "e4m3", "f32"])
@pytest.mark.parametrize("q_dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [2, 20, 64])
def test_maxima_that_keep_moving(tts, kv, q_dt, T):
    """Scores that grow along the window, within tiles and across them: every rescaling path."""
    hq, hkv, d, cap, past = 4, 2, 128, 900, 820
    c = R.Cache(1, hkv, d, cap, kv, 0, seed=8)
    ramp = torch.linspace(0.0, 6.0, cap)
    rng = np.random.default_rng(2)
    direction = torch.from_numpy(rng.standard_normal(d).astype(np.float32))
    direction /= direction.norm()
    rows = 0.2 * torch.from_numpy(rng.standard_normal((1, hkv, cap, d)).astype(np.float32)) + \
        (ramp * 8)[None, None, :, None] * direction
    c.k, c.ks = R.to_cache(rows.numpy(), kv)
    c.to_device(tts, hq)
    q = (direction + 0.05 * torch.from_numpy(rng.standard_normal((1, T, hq, d)).astype(np.float32))).to(R.TORCH[q_dt])
    m = masks(1, T, 3)
    out, _ = run_tree(tts, c, q.cuda(), [past], [T], m, T, 1.0)
    ref, mag = R.tree_attn(c, q.double(), [past], [T], m, 1.0)
    # scores of up to 50: their f32 sums (2^-24 of a sum of magnitudes of about 60, a few
    # roundings) move a weight by up to 2e-5 of itself; a weight whose tile's maximum moved after
    # it was written is rounded a second time
    bound = 4e-5 * mag + 1e-5 * ref.abs().amax(-1, keepdim=True)
    if q_dt == "bf16":
        bound = bound + 2.0 ** -8 * ref.abs() + 2.0 ** -7 * mag
    assert ((out.cpu().double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("kv", ["i8", "e4m3"])
@pytest.mark.parametrize("q_dt", ["bf16", "f32"])
def test_scales_and_queries_of_all_sizes(tts, kv, q_dt):
    """Row scales from 2^-60 to 2^60 (also negative ones and zero rows), query rows from 2^-90 to
    2^30 and of zeros: what the f16 operands' powers of two have to follow."""
    T, hq, hkv, d, cap, past = 8, 4, 2, 128, 1200, 1100
    rng = np.random.default_rng(4)
    for case in range(4):
        c = R.Cache(1, hkv, d, cap, kv, 0, seed=9 + case)
        if case == 0:      # V scales that grow, fall and jump from tile to tile
            e = np.repeat(rng.integers(-60, 60, (cap + 99) // 100), 100)[:cap]
        elif case == 1:    # and from row to row
            e = rng.integers(-20, 20, cap)
        else:
            e = np.full(cap, -100 if case == 2 else 100)
        c.vs *= torch.from_numpy(np.exp2(e).astype(np.float32))
        c.vs[:, :, ::7] *= -1
        c.ks[:, :, ::5] *= -1
        c.vs[:, :, 3::11] = 0
        c.ks[:, :, 4::13] = 0
        c.to_device(tts, hq)
        q = torch.from_numpy(rng.standard_normal((1, T, hq, d)).astype(np.float32))
        q *= torch.from_numpy(np.exp2(np.array([0, -90, 0, -3, 2, 0, -20, 1])).astype(np.float32))[None, :, None, None]
        q[0, 2] = 0
        q = q.to(R.TORCH[q_dt])
        for scale in (0.09, 0.0):
            out, _ = run_tree(tts, c, q.cuda(), [past], [T], None, T, scale)
            check_tree(out, *R.tree_attn(c, q.double(), [past], [T], None, scale), [T])
    # one row of q so large that the scores need its power of two: all weight on the best row
    q = torch.from_numpy(rng.standard_normal((1, T, hq, d)).astype(np.float32) * 2.0 ** 30).to(R.TORCH[q_dt])
    out, _ = run_tree(tts, c, q.cuda(), [past], [T], None, T, 2.0 ** -30 * 0.09)
    check_tree(out, *R.tree_attn(c, q.double(), [past], [T], None, 2.0 ** -30 * 0.09), [T])


@pytest.mark.parametrize("q_dt", ["bf16", "f32"])
def test_codes_that_are_not_numbers(tts, q_dt):
    # e4m3 NaN codes (which writing never makes) in rows that only some nodes see
    T, hq, hkv, d, cap, past = 6, 2, 1, 128, 400, 300
    c = R.Cache(1, hkv, d, cap, "e4m3", 0, seed=3)
    c.v.view(torch.uint8)[0, 0, past + 2, 9] = 0x7F
    c.k.view(torch.uint8)[0, 0, past + 4, 0] = 0xFF
    c.to_device(tts, hq)
    m = np.array([[1, 3, 7, 1 | 8, 1 | 16, 1 | 32]], np.int64)
    q = torch.randn(1, T, hq, d, generator=torch.Generator().manual_seed(1)).to(R.TORCH[q_dt])
    out, _ = run_tree(tts, c, q.cuda(), [past], [T], m, T, 0.1)
    ref, mag = R.tree_attn(c, q.double(), [past], [T], m, 0.1)
    o = out.cpu()
    assert o[0, 2, :, 9].isnan().all() and o[0, 4].isnan().all()
    keep = [i for i in range(d) if i != 9]
    check_tree(out[:, :4][..., keep], ref[:, :4][..., keep], mag[:, :4][..., keep], [4])
    check_tree(out[:, [0, 1, 3, 5]], ref[:, [0, 1, 3, 5]], mag[:, [0, 1, 3, 5]], [4])


@pytest.mark.parametrize("kv,q_dt", [("i8", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
def test_row_blocks_beyond_the_nodes(tts, kv, q_dt):
    # 64 nodes of 4 q heads are several row blocks; a stream with few nodes leaves some empty
    B, T, hq, hkv, d, cap = 3, 64, 4, 1, 64, 1500
    past, nodes = [1300, 40, 700], [64, 5, 33]
    c = R.Cache(B, hkv, d, cap, kv, 0, seed=2, fill=[p + n for p, n in zip(past, nodes)]).to_device(tts, hq)
    q = torch.randn(B, T, hq, d, generator=torch.Generator().manual_seed(5)).to(R.TORCH[q_dt])
    out, ef = run_tree(tts, c, q.cuda(), past, nodes, None, T, 0.125)
    assert ef == 0
    check_tree(out, *R.tree_attn(c, q.double(), past, nodes, None, 0.125), nodes)
    for b in range(B):
        assert (out[b, nodes[b]:] == 9).all()


def test_two_graphs_that_share_a_workspace_take_turns(tts):
    # each graph is captured over one workspace; replayed one after the other on one stream, each
    # gives its own result
    B, T, hq, hkv, d, cap = 2, 4, 4, 2, 128, 3000
    g = torch.Generator().manual_seed(6)
    caches = [R.Cache(B, hkv, d, cap, "i8", 0, seed=s, fill=[2500, 2900]).to_device(tts, hq) for s in (1, 2)]
    qs = [torch.randn(B * T, hq * d, generator=g).bfloat16().cuda() for _ in range(2)]
    past = ints([2496, 2896])
    ws = tts.tree_workspace(caches[0].desc, T, torch.bfloat16)
    outs = [torch.empty(B, T, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    eager = []
    for c, q, o in zip(caches, qs, outs):
        tts.tts_tree_attn(q, c.cache, c.desc, past, T, 0.1, o, ws)
        eager.append(o.clone())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        for c, q, o in zip(caches, qs, outs):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=s):
                tts.tts_tree_attn(q, c.cache, c.desc, past, T, 0.1, o, ws)
            graphs.append(gr)
        for o in outs:
            o.zero_()
        for _ in range(20):
            graphs[0].replay()
            graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], eager[0]) and torch.equal(outs[1], eager[1])


# ---------------------------------------------------------------------------
# Commit
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kv,d,page", [("f32", 128, 0), ("bf16", 64, 16), ("i8", 128, 1), ("e4m3", 64, 0), ("i8", 64, 64),
                                       ("bf16", 128, 4)])
@pytest.mark.parametrize("T", [1, 9, 64])
def test_commit(tts, kv, d, page, T):
    B, hkv, cap = 5, 3, 256
    rng = np.random.default_rng(T)
    c = R.Cache(B, hkv, d, cap, kv, page, seed=T).to_device(tts, 2 * hkv)
    n = [0, min(1, T), T, max(1, T // 2), max(1, T // 3)]
    past = [0, 3, cap - T, 60, 100]
    path = np.full((B, T), 10 ** 6, np.int32)     # entries past n_accept are not looked at
    for b in range(B):
        path[b, :n[b]] = np.sort(rng.permutation(T)[:n[b]])
    ef = flag()
    wide = torch.zeros(B, T + 3, dtype=I32, device="cuda")
    wide[:, :T] = torch.from_numpy(path).cuda()
    tts.tts_tree_commit(c.cache, c.desc, ints(past), wide[:, :T], ints(n), T, err_flag=ef)
    assert ef.item() == 0
    for t in [c.k, c.v] + ([c.ks, c.vs] if c.ks is not None else []):
        t = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
        old = t.clone()
        for b in range(B):
            for i in range(n[b]):
                sa, sr = c.at(b, past[b] + int(path[b, i]))
                da, dr = c.at(b, past[b] + i)
                t[da, :, dr] = old[sa, :, sr]
    assert all(torch.equal(a, b) for a, b in zip(c.back(), c.host()))


def test_commit_refuses_bad_paths(tts):
    B, T = 8, 6
    c = R.Cache(B, 2, 64, 64, "i8", 16, seed=1)
    c.bt[6, 2] = -7
    c.to_device(tts, 4)
    path = ints([[2, 1, 0, 0, 0, 0], [0, 0, 1, 2, 3, 4], [0, 6, 0, 0, 0, 0], [-1, 2, 0, 0, 0, 0], [0, 1, 2, 3, 4, 5],
                 [0, 5, 0, 0, 0, 0], [0, 5, 0, 0, 0, 0], [1, 3, 0, 0, 0, 0]])
    n, past = [2, 3, 2, 2, 7, 2, 2, 2], [0, 0, 0, 0, 0, 59, 30, -1]
    expect = [tts.EFLAG_ID_RANGE] * 5 + [tts.EFLAG_POS_RANGE, tts.EFLAG_PAGE, tts.EFLAG_POS_RANGE]
    for b in range(B):
        nn = [0] * B
        nn[b] = n[b]
        ef = flag()
        tts.tts_tree_commit(c.cache, c.desc, ints(past), path, ints(nn), T, err_flag=ef)
        assert ef.item() == expect[b], b
        assert all(torch.equal(x, y) for x, y in zip(c.back(), c.host())), b


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
class Loop:
    """Drafted decoding of B streams, as a program would run it: draft rows rotated, written
    and attended, the accepted path committed, the next token decoded."""

    def __init__(self, tts, kv, page, q_dt, seed):
        self.tts = tts
        self.B, self.T, self.hq, self.hkv, self.d, self.cap = 3, 7, 8, 4, 128, 512
        self.past = [0, 100, 400]
        self.c = R.Cache(self.B, self.hkv, self.d, self.cap, kv, page, seed=seed).to_device(tts, self.hq)
        g = torch.Generator().manual_seed(seed)
        n, w = self.B * self.T, (self.hq + 2 * self.hkv) * self.d
        self.x = torch.randn(n, w, generator=g)
        self.rng = np.random.default_rng(seed)
        self.mask = np.stack([R.random_tree(self.T, self.rng) for _ in range(self.B)])
        self.depth = np.array([[bin(int(m)).count("1") - 1 for m in row] for row in self.mask])
        self.cs = torch.from_numpy(R.table(600, 64, 1e4, kind="linear", factor=2.0)).float().contiguous()
        self.gq, self.gk = torch.rand(self.d, generator=g) + 0.5, torch.rand(self.d, generator=g) + 0.5
        self.path = np.zeros((self.B, self.T), np.int32)
        self.n_acc = []
        for b in range(self.B):
            leaf = int(np.argmax(self.depth[b]))
            nodes = [u for u in range(self.T) if int(self.mask[b, leaf]) >> u & 1]
            self.path[b, :len(nodes)] = nodes
            self.n_acc.append(len(nodes))
        self.q_dt = R.TORCH[q_dt]
        dev = "cuda"
        self.d_x, self.d_cs, self.d_gq, self.d_gk = (t.to(dev) for t in (self.x, self.cs, self.gq, self.gk))
        self.d_mask, self.d_path = torch.from_numpy(self.mask).to(dev), torch.from_numpy(self.path).to(dev)
        self.d_past, self.d_acc = ints(self.past), ints(self.n_acc)
        self.d_pos = (self.d_past[:, None] + torch.from_numpy(self.depth).to(dev).to(I32)).reshape(-1).contiguous()
        self.qr = torch.empty(n, self.hq * self.d, dtype=self.q_dt, device=dev)
        self.kr = torch.empty(n, self.hkv * self.d, dtype=self.q_dt, device=dev)
        self.vr = self.d_x[:, -self.hkv * self.d:].to(self.q_dt).contiguous()   # k and v share a stride
        self.out = torch.empty(self.B, self.T, self.hq, self.d, dtype=self.q_dt, device=dev)
        self.last = torch.empty(self.B, self.hq, self.d, dtype=self.q_dt, device=dev)
        self.ws = tts.tree_workspace(self.c.desc, self.T, self.q_dt)
        self.ef = flag()
        self.scale = self.d ** -0.5

    def step(self):
        t, c, qd, kd = self.tts, self.c, self.hq * self.d, self.hkv * self.d
        t.tts_rope_rows(self.d_x[:, :qd], self.d_x[:, qd:qd + kd], self.qr, self.kr, self.d_pos, self.hq, self.hkv, self.d,
                        self.d_cs, gamma_q=self.d_gq, gamma_k=self.d_gk, interleaved=True, err_flag=self.ef)
        t.tts_kv_write_rows(self.kr, self.vr, c.cache, c.desc, self.d_past, self.T, err_flag=self.ef)
        t.tts_tree_attn(self.qr, c.cache, c.desc, self.d_past, self.T, self.scale, self.out, self.ws,
                        tree_mask=self.d_mask, err_flag=self.ef)
        t.tts_tree_commit(c.cache, c.desc, self.d_past, self.d_path, self.d_acc, self.T, err_flag=self.ef)
        # the first node's query again, over the committed window (its last row as the node)
        t.tts_tree_attn(self.qr.view(self.B, self.T, qd)[:, 0], c.cache, c.desc, self.d_past + self.d_acc - 1, 1,
                        self.scale, self.last, self.ws, err_flag=self.ef)

    def check(self):
        assert self.ef.item() == 0
        c, B, T, d = self.c, self.B, self.T, self.d
        pos = self.d_pos.cpu()
        x = self.x.double()
        qd, kd = self.hq * d, self.hkv * d
        qr = R.rope(x[:, :qd].reshape(B * T, self.hq, d), pos, self.cs, 64, True, self.gq)
        tol = 2.0 ** -8 if self.q_dt == torch.bfloat16 else 0.0
        assert ((self.qr.cpu().double().reshape(qr.shape) - qr).abs() <= tol * qr.abs() + 2e-6 * qr.abs().amax()).all()
        # the rows as the device rounded them, through the definitions
        for which, rows in ((0, self.kr), (1, self.vr)):
            code, s = R.to_cache(rows.cpu().float().reshape(B * T, self.hkv, d).numpy(), c.kv)
            t, sc = (c.k, c.ks) if which == 0 else (c.v, c.vs)
            for b in range(B):
                for i in range(T):
                    at, row = c.at(b, self.past[b] + i)
                    t[at, :, row] = code[b * T + i]
                    if sc is not None:
                        sc[at, :, row] = s[b * T + i]
        q = self.qr.cpu().double().reshape(B, T, self.hq, d)
        check_tree(self.out, *R.tree_attn(c, q, self.past, [T] * B, self.mask, self.scale), [T] * B)
        for t in [c.k, c.v] + ([c.ks, c.vs] if c.ks is not None else []):
            t = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
            old = t.clone()
            for b in range(B):
                for i in range(self.n_acc[b]):
                    sa, sr = c.at(b, self.past[b] + int(self.path[b, i]))
                    da, dr = c.at(b, self.past[b] + i)
                    t[da, :, dr] = old[sa, :, sr]
        assert all(torch.equal(a, b) for a, b in zip(c.back(), c.host()))
        end = [p + n - 1 for p, n in zip(self.past, self.n_acc)]
        check_tree(self.last[:, None], *R.tree_attn(c, q[:, :1], end, [1] * B, None, self.scale), [1] * B)


@pytest.mark.parametrize("kv,page,q_dt", [("i8", 16, "bf16"), ("e4m3", 0, "bf16"), ("bf16", 64, "bf16"), ("f32", 0, "f32"),
                                          ("i8", 0, "f32")])
def test_a_drafted_step(tts, kv, page, q_dt):
    loop = Loop(tts, kv, page, q_dt, 11)
    loop.step()
    loop.check()


@pytest.mark.parametrize("kv,q_dt", [("i8", "bf16"), ("bf16", "bf16"), ("f32", "f32")])
def test_a_drafted_step_in_a_graph(tts, kv, q_dt):
    loop, eager = Loop(tts, kv, 16, q_dt, 12), Loop(tts, kv, 16, q_dt, 12)
    eager.step()
    before = [t.clone() for t in (loop.c.dk, loop.c.dv, loop.c.dks, loop.c.dvs) if t is not None]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        loop.step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            loop.step()
    for _ in range(2):
        for t, old in zip([t for t in (loop.c.dk, loop.c.dv, loop.c.dks, loop.c.dvs) if t is not None], before):
            t.copy_(old)
        loop.out.zero_()
        loop.last.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loop.out, eager.out) and torch.equal(loop.last, eager.last)
        assert all(torch.equal(a, b) for a, b in zip(loop.c.back(), eager.c.back()))


def test_two_streams_at_once(tts):
    a, b = Loop(tts, "i8", 16, "bf16", 13), Loop(tts, "i8", 16, "bf16", 14)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for s, loop in ((sa, a), (sb, b)):
        with torch.cuda.stream(s):
            loop.step()
    torch.cuda.synchronize()
    a.check()
    b.check()
