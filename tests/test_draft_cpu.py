"""Refusals of the drafted-decoding calls (tts_rope_rows, tts_kv_write_rows, tts_tree_attn and
their kin) before any launch, the checks of the binding, and the host plans.  No GPU."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import draft_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only validation checks")


@pytest.fixture(scope="module")
def tts():
    from autoregressive_codebook_tts_gb300 import build
    build.build()
    from autoregressive_codebook_tts_gb300 import tts as mod
    return mod


def ptr(x):
    return P(x) if x else None


def cache_of(tts, k=256, v=256, ks=256, vs=256):
    return tts.TtsKvCache(k or None, v or None, ks or None, vs or None)


def test_constants_match_the_header(tts):
    src = open(os.path.join(ROOT, "include", "tts_decode.h")).read()
    dt = dict(re.findall(r"(TTS_I8|TTS_E4M3) = (\d+)", src))
    assert (tts.TTS_I8, tts.TTS_E4M3) == (int(dt["TTS_I8"]), int(dt["TTS_E4M3"]))
    assert tts.TTS_MAX_TREE_NODES == int(re.search(r"#define TTS_MAX_TREE_NODES (\d+)", src).group(1))
    kinds = dict(re.findall(r"TTS_ROPE_(NONE|LINEAR|BASE|PARTS) = (\d)", src))
    assert tts._ROPE_KINDS == {k.lower(): int(v) for k, v in kinds.items()}


@no_gpu
def test_the_earlier_calls_refuse_8_bit_caches(tts):
    for kv in ("i8", "e4m3"):
        d = tts.kv_desc(1, 16, 8, 128, 256, kv)
        assert tts.tts_decode_attn_workspace_size(d, 1) == 0
        assert tts._lib.tts_kv_set_rows(P(16), P(16), 1024, P(16), P(16), ctypes.byref(d), P(16), None, None) == 3
        assert tts.tts_prefill_workspace_size(d, 4, 0) == 0


@no_gpu
def test_rope_table_scaled_refuses(tts):
    def call(cs=16, n=64, rot=64, base=1e6, kind=0, L=64, f=2.0, lo=1.0, hi=32.0, a=1.0, s=True):
        sc = tts.TtsRopeScaling(kind, L, f, lo, hi, a)
        return tts._lib.tts_rope_table_scaled(ptr(cs), n, rot, base, ctypes.byref(sc) if s else None, None)
    assert call(cs=0) == 1 and call(s=False) == 1
    assert call(kind=4) == 3 and call(kind=-1) == 3
    for bad in (dict(n=0), dict(n=(1 << 26) + 1), dict(rot=0), dict(rot=63), dict(rot=130), dict(base=1.0),
                dict(base=float("inf")), dict(base=float("nan")), dict(a=0.0), dict(a=float("inf")),
                dict(kind=1, f=0.5), dict(kind=1, f=float("nan")), dict(kind=2, rot=2), dict(kind=2, f=float("inf")),
                dict(kind=3, L=0), dict(kind=3, lo=-1.0), dict(kind=3, lo=32.0), dict(kind=3, hi=float("inf"))):
        assert call(**bad) == 2, bad
    assert call(cs=8) == 5


@no_gpu
def test_rope_rows_refuses(tts):
    def call(q=16, k=16, qo=32, ko=32, qs=2048, ks=1024, qos=2048, kos=1024, dt=0, odt=0, gq=16, gk=16, eps=1e-6,
             pos=16, rows=4, hq=16, hkv=8, d=128, rot=128, inter=0, cs=16, n=64):
        return tts._lib.tts_rope_rows(ptr(q), qs, ptr(k), ks, dt, ptr(qo), qos, ptr(ko), kos, odt, ptr(gq), ptr(gk),
                                      eps, ptr(pos), rows, hq, hkv, d, rot, inter, ptr(cs), n, None, None)
    for bad in (dict(q=0), dict(k=0), dict(qo=0), dict(ko=0), dict(pos=0), dict(cs=0), dict(gq=0), dict(gk=0)):
        assert call(**bad) == 1, bad
    assert call(dt=2) == 3 and call(odt=3) == 3
    for bad in (dict(rows=0), dict(rows=(1 << 24) + 1), dict(d=96), dict(hq=0), dict(hkv=-1), dict(rot=0), dict(rot=3),
                dict(rot=130), dict(n=0), dict(eps=-1.0), dict(eps=float("nan")), dict(inter=2), dict(qs=2044),
                dict(kos=1020)):
        assert call(**bad) == 2, bad
    for bad in (dict(q=24), dict(ko=40), dict(cs=24), dict(gk=8), dict(qs=2050), dict(odt=1, qos=2052)):
        assert call(**bad) == 5, bad
    assert call(qo=16, odt=1) == 4                # in place with another type
    assert call(ko=16, kos=1028) == 4             # in place with another stride


@no_gpu
def test_kv_rows_refuse(tts):
    def call(read, k=16, v=16, dt=0, stride=1024, c=None, d=None, start=16, T=4, with_cache=True):
        d = tts.kv_desc(2, 16, 8, 128, 256, "i8") if d is None else d
        c = cache_of(tts) if c is None else c
        cp = ctypes.byref(c) if with_cache else None
        if read:
            return tts._lib.tts_kv_read_rows(cp, ctypes.byref(d), ptr(start), None, T, ptr(k), ptr(v), dt, stride, None, None)
        return tts._lib.tts_kv_write_rows(ptr(k), ptr(v), dt, stride, cp, ctypes.byref(d), ptr(start), None, T, None, None)
    for read in (False, True):
        assert call(read, k=0) == 1 and call(read, v=0) == 1 and call(read, start=0) == 1
        assert call(read, with_cache=False) == 1
        for c in (dict(k=0), dict(v=0), dict(ks=0), dict(vs=0)):
            assert call(read, c=cache_of(tts, **c)) == 1, c
        assert call(read, c=cache_of(tts, k=264)) == 5 and call(read, c=cache_of(tts, vs=260)) == 5
        assert call(read, dt=2) == 3 and call(read, dt=3) == 3
        assert call(read, T=0) == 2 and call(read, T=(1 << 24)) == 2 and call(read, stride=1000) == 2
        assert call(read, stride=1026) == 5 and call(read, dt=1, stride=1028) == 5
        assert call(read, k=24) == 5 and call(read, v=24) == 5
        assert call(read, d=tts.kv_desc(2, 16, 8, 96, 256, "i8")) == 2
        bad = tts.kv_desc(2, 16, 8, 128, 256, "i8")
        bad.kv_dtype = 2                          # Q8_0 is a table format
        assert call(read, d=bad) == 3
        assert call(read, d=tts.kv_desc(2, 16, 8, 128, 256, "i8", paged=True, page_size=16, n_pages=4)) == 1


@no_gpu
def test_tree_attn_refuses(tts):
    def call(q=16, qdt=0, qs=2048, c=None, d=None, past=16, mask=16, T=8, scale=0.1, out=16, ws=256, ws_bytes=1 << 30):
        d = tts.kv_desc(2, 16, 8, 128, 4096, "bf16") if d is None else d
        c = cache_of(tts) if c is None else c
        return tts._lib.tts_tree_attn(ptr(q), qdt, qs, ctypes.byref(c), ctypes.byref(d), ptr(past), None, ptr(mask), T,
                                      scale, ptr(out), ptr(ws), ws_bytes, None, None)
    for bad in (dict(q=0), dict(past=0), dict(out=0)):
        assert call(**bad) == 1, bad
    assert call(qdt=2) == 3 and call(qdt=3) == 3
    for bad in (dict(T=0), dict(T=65), dict(qs=2044), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(d=tts.kv_desc(2, 16, 3, 128, 4096, "bf16")), dict(d=tts.kv_desc(70000, 16, 8, 128, 4096, "bf16"))):
        assert call(**bad) == 2, bad
    for bad in (dict(q=24), dict(out=24), dict(mask=24), dict(qs=2050), dict(qdt=1, qs=2052), dict(ws=272)):
        assert call(**bad) == 5, bad
    assert call(ws=0) == 6 and call(ws_bytes=1024) == 6
    d = tts.kv_desc(2, 16, 8, 128, 4096, "bf16")
    for dt in ("f32", "bf16"):
        assert tts.tts_tree_attn_workspace_size(d, 8, dt) > 0
    assert tts.tts_tree_attn_workspace_size(d, 65) == 0 and tts.tts_tree_attn_workspace_size(d, 0) == 0


@no_gpu
def test_tree_commit_refuses(tts):
    def call(c=None, past=16, path=16, stride=8, n=16, T=8):
        d = tts.kv_desc(2, 16, 8, 128, 256, "e4m3")
        c = cache_of(tts) if c is None else c
        return tts._lib.tts_tree_commit(ctypes.byref(c), ctypes.byref(d), ptr(past), ptr(path), stride, ptr(n), T, None, None)
    assert call(past=0) == 1 and call(path=0) == 1 and call(n=0) == 1 and call(c=cache_of(tts, ks=0)) == 1
    assert call(T=0) == 2 and call(T=65, stride=65) == 2 and call(stride=7) == 2


def test_binding_refuses_what_the_library_cannot_see(tts):
    k = torch.zeros(2, 8, 256, 128, dtype=torch.int8)
    s = torch.zeros(2, 8, 256)
    with pytest.raises(ValueError, match="scale"):
        tts.kv_cache(k, k)
    with pytest.raises(ValueError, match="scale"):
        tts.kv_cache(k.float(), k.float(), s, s)
    with pytest.raises(ValueError, match="one per cache row"):
        tts.kv_cache(k, k, s[:, :4], s)
    with pytest.raises(ValueError, match="contiguous"):
        tts.kv_cache(k.transpose(1, 2), k.transpose(1, 2), s, s)
    with pytest.raises(ValueError, match="dtype"):
        tts.kv_cache(k.to(torch.uint8), k.to(torch.uint8), s, s)
    c = tts.kv_cache(k, k, s, s)
    d = tts.kv_desc(2, 16, 8, 128, 256, "i8")
    rows = torch.zeros(4, 1024)
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="descriptor"):
        tts.tts_kv_write_rows(rows, rows, c, tts.kv_desc(2, 16, 8, 128, 512, "i8"), pos, 2)
    with pytest.raises(ValueError, match="descriptor"):
        tts.tts_kv_write_rows(rows, rows, c, tts.kv_desc(2, 16, 8, 128, 256, "e4m3"), pos, 2)
    with pytest.raises(ValueError, match="B \\* T"):
        tts.tts_kv_write_rows(rows, rows, c, d, pos, 3)
    with pytest.raises(ValueError, match="int32"):
        tts.tts_kv_write_rows(rows, rows, c, d, pos.long(), 2)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        tts.tts_kv_write_rows(rows.half(), rows.half(), c, d, pos, 2)
    with pytest.raises(ValueError, match="current CUDA device"):
        tts.tts_kv_write_rows(rows, rows, c, d, pos, 2)
    q = torch.zeros(4, 2048, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="out must be"):
        tts.tts_tree_attn(q, c, d, pos, 2, 0.1, q.float(), None)
    with pytest.raises(ValueError, match="int64"):
        tts.tts_tree_attn(q, c, d, pos, 2, 0.1, torch.empty_like(q), None, tree_mask=torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="path"):
        tts.tts_tree_commit(c, d, pos, torch.zeros(2, 3, dtype=torch.int32), pos, 2)
    with pytest.raises(ValueError, match="kind"):
        tts.tts_rope_table_scaled(torch.empty(4, 2, 2), 4, 4, 1e4, kind="other")
    with pytest.raises(ValueError, match="table"):
        tts.tts_rope_rows(rows, None, rows, None, torch.zeros(4, dtype=torch.int32), 8, 0, 128, torch.zeros(4, 64))


@no_gpu
def test_rope_table_scaled_refuses_more_rows_than_a_grid_holds(tts):
    # blocks of 1024 positions, at most 65535 of them
    sc = tts.TtsRopeScaling(0, 1, 1.0, 1.0, 32.0, 1.0)
    for n in (65535 * 1024 + 1, 1 << 26):
        assert tts._lib.tts_rope_table_scaled(P(16), n, 64, 1e6, ctypes.byref(sc), None) == 2, n


@no_gpu
def test_tree_attn_refuses_scales_that_overflow_in_base_2(tts):
    d, c = tts.kv_desc(2, 16, 8, 128, 4096, "bf16"), cache_of(tts)
    for scale in (3e38, -3e38):   # times log2(e): beyond the largest f32
        assert tts._lib.tts_tree_attn(P(16), 0, 2048, ctypes.byref(c), ctypes.byref(d), P(16), None, None, 8, scale,
                                      P(1 << 20), P(256), 1 << 30, None, None) == 2, scale


@no_gpu
def test_tree_attn_refuses_out_over_q(tts):
    d, c = tts.kv_desc(2, 16, 8, 128, 4096, "bf16"), cache_of(tts)
    for q_dtype in (0, 1):
        assert tts._lib.tts_tree_attn(P(1 << 20), q_dtype, 2048, ctypes.byref(c), ctypes.byref(d), P(16), None, None, 8,
                                      0.1, P(1 << 20), P(256), 1 << 30, None, None) == 4


def test_binding_refuses_small_flags_and_expanded_workspaces(tts):
    k, s = torch.zeros(2, 8, 256, 128, dtype=torch.int8), torch.zeros(2, 8, 256)
    c, d = tts.kv_cache(k, k, s, s), tts.kv_desc(2, 16, 8, 128, 256, "i8")
    rows, q, pos = torch.zeros(4, 1024), torch.zeros(4, 2048), torch.zeros(2, dtype=torch.int32)
    path, byte = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.uint8)
    ws = torch.zeros(1, dtype=torch.uint8).expand(1 << 20)
    calls = (lambda **kw: tts.tts_kv_write_rows(rows, rows, c, d, pos, 2, **kw),
             lambda **kw: tts.tts_kv_read_rows(c, d, pos, 2, rows, rows, **kw),
             lambda **kw: tts.tts_tree_attn(q, c, d, pos, 2, 0.1, torch.empty_like(q), None, **kw),
             lambda **kw: tts.tts_tree_commit(c, d, pos, path, pos, 2, **kw),
             lambda **kw: tts.tts_rope_rows(rows, None, torch.empty_like(rows), None, torch.zeros(4, dtype=torch.int32),
                                            8, 0, 128, torch.zeros(4, 64, 2), **kw))
    for call in calls:
        with pytest.raises(ValueError, match="err_flag"):
            call(err_flag=byte)
    with pytest.raises(ValueError, match="workspace"):
        tts.tts_tree_attn(q, c, d, pos, 2, 0.1, torch.empty_like(q), ws)


def test_descriptors_name_their_dtype(tts):
    # (an unknown name once meant bf16: two bytes an entry over a one-byte tensor)
    for names, code in ((("f32", "float32", torch.float32), tts.TTS_F32), (("bf16", "bfloat16", torch.bfloat16), tts.TTS_BF16),
                        (("i8", "int8", torch.int8), tts.TTS_I8),
                        (("e4m3", "float8_e4m3fn", torch.float8_e4m3fn), tts.TTS_E4M3)):
        for name in names:
            assert tts.kv_desc(1, 16, 8, 128, 256, name).kv_dtype == code, name
    for name in ("fp8", "int4", "f16", "", None, torch.float16, torch.uint8, torch.float8_e5m2):
        with pytest.raises(ValueError, match="kv_dtype"):
            tts.kv_desc(1, 16, 8, 128, 256, name)


def test_descriptors_check_their_block_table(tts):
    def desc(bt, B=2):
        return tts.kv_desc(B, 16, 8, 128, 256, "i8", paged=True, page_size=16, n_pages=40, block_table=bt)
    bt = torch.arange(32, dtype=torch.int32).reshape(2, 16)
    assert desc(bt).bt_stride == 16 and desc(torch.zeros(3, 20, dtype=torch.int32)[:, :16]).bt_stride == 20
    # 64-bit ids (read as pairs), too few rows (read past the end), other strides
    for bad in (bt.long(), bt[:1], bt[0], bt.reshape(16, 2).t()):
        with pytest.raises(ValueError, match="block_table"):
            desc(bad)
    k, sc = torch.zeros(40, 8, 16, 128, dtype=torch.int8), torch.zeros(40, 8, 16)
    c, d = tts.kv_cache(k, k, sc, sc), desc(bt)
    d.table_device = 1
    rows = torch.zeros(4, 1024)
    with pytest.raises(ValueError, match="one device"):
        tts.tts_kv_write_rows(rows, rows, c, d, torch.zeros(2, dtype=torch.int32), 2)


# The reference's own quantiser against facts of the formats.
def test_reference_codes():
    assert R.E4M3.size == 127 and R.E4M3[-1] == 448.0 and R.E4M3[1] == 2.0 ** -9
    every = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(every, R.E4M3)
    x = np.array([0.5, 1.5, 2.5, -0.5, 126.5, 200.0])
    assert R.nearest_code(x, "i8").tolist() == [0, 2, 2, -0.0, 126, 127]
    # halfway between 1 and 1.125, 1.125 and 1.25; the smallest two
    assert R.nearest_code(np.array([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10]), "e4m3").tolist() == [
        1.0, 1.25, 0.0, 2.0 ** -8]
