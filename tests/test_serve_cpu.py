"""Refusals of the calls that serve many requests at once (tts_add_rms_norm, tts_project_rows,
tts_page_plan, tts_kv_write_slots) before any launch, and the checks of the binding.  No GPU."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only validation checks")
OK, NULL, SHAPE, DTYPE, LAYOUT, ALIGN, WORKSPACE = range(7)


@pytest.fixture(scope="module")
def tts():
    from autoregressive_codebook_tts_gb300 import build
    build.build()
    from autoregressive_codebook_tts_gb300 import tts as mod
    return mod


def ptr(x):
    return P(x) if x else None


def test_constants_match_the_header(tts):
    src = open(os.path.join(ROOT, "include", "tts_decode.h")).read()
    for name in ("TTS_MAX_NORM_WIDTH", "TTS_MAX_ADAPTER_RANK", "TTS_MAX_PLAN_STREAMS"):
        assert getattr(tts, name) == int(re.search(rf"#define {name} (\d+)", src).group(1))


@no_gpu
def test_add_rms_norm_refuses(tts):
    def call(x=16, xs=64, xd=0, r=32, rs=64, rd=0, s=48, ss=64, g=16, eps=1e-6, rows=4, n=64, o=64, os_=64, od=0, sc=0):
        return tts._lib.tts_add_rms_norm(ptr(x), xs, xd, ptr(r), rs, rd, ptr(s), ss, ptr(g), eps, rows, n, ptr(o), os_, od,
                                         ptr(sc), None)
    for bad in (dict(x=0), dict(g=0), dict(o=0), dict(od=4), dict(r=0)):
        assert call(**bad) == NULL, bad
    for bad in (dict(xd=2), dict(rd=4), dict(od=3), dict(xd=4)):
        assert call(**bad) == DTYPE, bad
    for bad in (dict(rows=0), dict(rows=(1 << 24) + 1), dict(n=0), dict(n=60), dict(n=16392, xs=16392, rs=16392, ss=16392, os_=16392),
                dict(eps=-1.0), dict(eps=float("nan")), dict(xs=60), dict(rs=60), dict(ss=60), dict(os_=60)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(x=24), dict(r=40), dict(s=56), dict(g=8), dict(o=72), dict(od=4, sc=8), dict(xs=66), dict(xd=1, xs=68),
                dict(od=4, sc=16, os_=68), dict(od=4, sc=16, o=68), dict(rd=1, rs=68), dict(rd=1, ss=68)):
        assert call(**bad) == ALIGN, bad
    # in place with another type or stride, or over another operand
    for bad in (dict(o=16, od=1), dict(o=16, os_=68), dict(s=32, ss=68), dict(o=32), dict(o=48), dict(s=16)):
        assert call(**bad) == LAYOUT, bad


def pool(tts, a=16, b=16, rank=16, scale=16, n=4, r=16):
    return tts.TtsAdapters(a or None, b or None, rank or None, scale or None, n, r)


@no_gpu
def test_project_rows_refuses(tts):
    def call(x=16, xs=64, dt=1, sx=0, w=32, sw=0, n=48, k=64, ad=True, rs=16, sa=16, ns=4, rows=4, o=64, os_=48, od=0, ws=256,
             wb=1 << 30):
        ad = pool(tts) if ad is True else ad
        return tts._lib.tts_project_rows(ptr(x), xs, dt, ptr(sx), ptr(w), ptr(sw), n, k, ctypes.byref(ad) if ad else None,
                                         ptr(rs), ptr(sa), ns, rows, ptr(o), os_, od, ptr(ws), wb, None, None)
    for bad in (dict(x=0), dict(w=0), dict(o=0), dict(dt=4), dict(dt=4, sx=16), dict(dt=4, sw=16), dict(sa=0),
                dict(ad=pool(tts, a=0)), dict(ad=pool(tts, b=0))):
        assert call(**bad) == NULL, bad
    for bad in (dict(dt=0), dict(dt=3), dict(od=4), dict(od=2)):
        assert call(**bad) == DTYPE, bad
    for bad in (dict(rows=0), dict(rows=(1 << 20) + 1), dict(n=0), dict(n=(1 << 20) + 1), dict(k=0), dict(k=65544), dict(xs=56),
                dict(os_=44), dict(ns=0), dict(ad=pool(tts, n=0)), dict(ad=pool(tts, r=0)), dict(ad=pool(tts, r=12)),
                dict(ad=pool(tts, r=136)), dict(ad=pool(tts, n=(1 << 31) - 1))):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(x=24), dict(w=40), dict(o=72), dict(xs=68), dict(k=60), dict(rs=10), dict(sa=10),
                dict(ad=pool(tts, a=24)), dict(ad=pool(tts, b=24)), dict(ad=pool(tts, rank=8)), dict(ad=pool(tts, scale=8)),
                dict(dt=4, sx=16, sw=16, k=72, xs=80), dict(dt=4, sx=8, sw=16), dict(dt=4, sx=16, sw=16, xs=72), dict(ws=128)):
        assert call(**bad) == ALIGN, bad
    assert call(ws=0) == WORKSPACE and call(wb=16) == WORKSPACE
    assert call(o=16, os_=64) == LAYOUT and call(o=32) == LAYOUT


@no_gpu
def test_page_plan_refuses(tts):
    d0 = dict(B=2, n_q_heads=16, n_kv_heads=8, head_dim=128, capacity=64, window_quantum=64, kv_dtype=1, paged=1, page_size=16,
              n_pages=9, bt_stride=4, flags=0, block_table=256)
    args = ["table", "free", "n_free", "past", "new", "T", "max_rows", "n_rows", "start", "stream", "pos", "slot"]

    def call(desc=None, **kw):
        v = dict({a: 256 for a in args}, T=0, max_rows=64)
        v.update(kw)
        d = tts.TtsKvDesc(**dict(d0, **(desc or {})))
        return tts._lib.tts_page_plan(ctypes.byref(d), *[v[a] if a in ("T", "max_rows") else ptr(v[a]) for a in args], None, None)
    for a in ("free", "n_free", "past", "new", "n_rows", "start", "stream", "pos", "slot"):
        assert call(**{a: 0}) == NULL, a
        assert call(**{a: 260 if a == "slot" else 258}) == ALIGN, a
    assert tts._lib.tts_page_plan(None, *[P(256)] * 5, 0, 64, *[P(256)] * 5, None, None) == NULL
    assert call(table=512) == LAYOUT and call(desc=dict(paged=0)) == LAYOUT
    assert call(desc=dict(block_table=None), table=0) == NULL
    assert call(desc=dict(page_size=12)) == LAYOUT and call(desc=dict(bt_stride=3)) == LAYOUT
    for bad in (dict(T=-1), dict(max_rows=0), dict(max_rows=(1 << 24) + 1), dict(T=8), dict(desc=dict(B=4097)),
                dict(desc=dict(n_pages=(1 << 30) + 1))):
        assert call(**bad) == SHAPE, bad


@no_gpu
def test_kv_write_slots_refuses(tts):
    def call(k=16, v=16, dt=0, stride=1024, c=None, d=None, slot=16, rows=4, with_cache=True):
        d = tts.kv_desc(2, 16, 8, 128, 256, "i8") if d is None else d
        c = tts.TtsKvCache(256, 256, 256, 256) if c is None else c
        return tts._lib.tts_kv_write_slots(ptr(k), ptr(v), dt, stride, ctypes.byref(c) if with_cache else None, ctypes.byref(d),
                                           ptr(slot), rows, None, None)
    for bad in (dict(k=0), dict(v=0), dict(slot=0), dict(with_cache=False), dict(c=tts.TtsKvCache(256, 256, None, 256)),
                dict(c=tts.TtsKvCache(None, 256, 256, 256))):
        assert call(**bad) == NULL, bad
    assert call(dt=2) == DTYPE and call(dt=4) == DTYPE
    for bad in (dict(rows=0), dict(rows=(1 << 24) + 1), dict(stride=1020), dict(d=tts.kv_desc(2, 16, 8, 96, 256, "i8"))):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(k=24), dict(v=24), dict(slot=12), dict(stride=1026), dict(dt=1, stride=1028),
                dict(c=tts.TtsKvCache(264, 256, 256, 256)), dict(c=tts.TtsKvCache(256, 256, 256, 264))):
        assert call(**bad) == ALIGN, bad


def test_binding_refuses_what_pointers_cannot_show(tts):
    f, h, q = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64).to(torch.float8_e4m3fn)
    g, sc = torch.ones(64), torch.zeros(4)
    norm = [dict(x=f[0]), dict(x=f.double()), dict(residual=f[:3]), dict(s=h), dict(gamma=g[:32]), dict(gamma=g.double()),
            dict(out=torch.zeros(4, 128)[:, ::2]), dict(out=q), dict(sc=sc), dict(out=q, sc=sc[:3]), dict(residual=None),
            dict(out=torch.zeros(5, 64)), dict()]
    for kw in norm:   # (the last is well formed, and refused for lying on the CPU)
        v = dict(dict(x=f, residual=f, s=f.clone(), gamma=g, out=f.clone(), sc=None), **kw)
        with pytest.raises(ValueError):
            tts.tts_add_rms_norm(v["x"], v["residual"], v["s"], v["gamma"], 1e-6, v["out"], out_scale=v["sc"])

    a, b = torch.zeros(3, 8, 64, dtype=torch.bfloat16), torch.zeros(3, 16, 8, dtype=torch.bfloat16)
    for bad in ((a.float(), b), (a[:2], b), (a, b.transpose(1, 2)), (a[:, :, :32], b), (a, b, torch.zeros(2, dtype=torch.int32)),
                (a, b, None, torch.zeros(3, dtype=torch.float64)), (a, b, torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(ValueError):
            tts.adapters(*bad)
    pool = tts.adapters(a, b)
    assert (pool.n, pool.k, pool.n_adapters, pool.rank_max) == (16, 64, 3, 8)
    w, of, ws = torch.zeros(16, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    other = tts.adapters(a, torch.zeros(3, 24, 8, dtype=torch.bfloat16))
    wq = torch.zeros(16, 64).to(torch.float8_e4m3fn)
    proj = [dict(x=f), dict(w=w[:, :32]), dict(w=w.T), dict(out=torch.zeros(4, 15)), dict(out=torch.zeros(4, 16).double()),
            dict(pool=other), dict(sa=None), dict(sa=of[:3]), dict(sa=of.long()), dict(rs=of[:3]), dict(rs=of.long()),
            dict(xs=sc), dict(ws_=sc), dict(x=q, w=wq), dict(x=q, w=wq, xs=sc[:2], ws_=torch.zeros(16)),
            dict(x=q, w=w, xs=sc, ws_=torch.zeros(16)), dict(work=torch.zeros(512, dtype=torch.uint8)[::2]), dict()]
    for kw in proj:
        v = dict(dict(x=h, w=w, out=torch.zeros(4, 16), work=ws, pool=pool, sa=of, rs=None, xs=None, ws_=None), **kw)
        with pytest.raises(ValueError):
            tts.tts_project_rows(v["x"], v["w"], v["out"], v["work"], x_scale=v["xs"], w_scale=v["ws_"], adapters=v["pool"],
                                 stream_adapter=v["sa"], row_stream=v["rs"])
    with pytest.raises(ValueError):
        tts.tts_project_workspace_size(4, 16, 64, "f32", pool)
    assert tts.tts_project_workspace_size(4, 16, 64, "bf16", None) == 0
    assert tts.tts_project_workspace_size(4, 16, 60, "bf16", pool) == 0

    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    tab = torch.zeros(2, 4, dtype=torch.int32)
    d = tts.kv_desc(2, 16, 8, 128, 64, "bf16", window_quantum=64, paged=True, page_size=16, n_pages=9, block_table=tab)
    ok = dict(tab=tab, free=i(9), nf=i(1), past=i(2), new=i(2), nr=i(2), start=i(3), stream=i(8), pos=i(8),
              slot=torch.zeros(8, dtype=torch.int64))
    for kw in (dict(tab=tab.clone()), dict(free=i(8)), dict(past=i(1)), dict(new=i(2).long()), dict(start=i(2)), dict(pos=i(7)),
               dict(slot=i(8)), dict(stream=i(16)[::2]), dict()):
        v = dict(ok, **kw)
        with pytest.raises(ValueError):
            tts.tts_page_plan(d, v["tab"], v["free"], v["nf"], v["past"], v["new"], v["nr"], v["start"], v["stream"], v["pos"],
                              v["slot"])

    kv = torch.zeros(9, 8, 16, 128, dtype=torch.bfloat16)
    cache, rows = tts.kv_cache(kv, kv.clone()), torch.zeros(4, 1024)
    for kw in (dict(k=rows[:3]), dict(v=rows.bfloat16()), dict(k=rows[:, :512]), dict(slot=i(4)),
               dict(slot=torch.zeros(3, dtype=torch.int64)), dict(d=tts.kv_desc(2, 16, 8, 128, 64, "f32", window_quantum=64)), dict()):
        v = dict(dict(k=rows, v=rows, slot=torch.zeros(4, dtype=torch.int64), d=d), **kw)
        with pytest.raises(ValueError):
            tts.tts_kv_write_slots(v["k"], v["v"], cache, v["d"], v["slot"])
