"""The calls that serve many requests at once against 64-bit restatements (serve_ref): the
residual's addition with the norm, projections with every row's own adapter, pages and row maps
from request lengths, rows written by slot -- alone, refused, poisoned, in graphs and on two
streams, and a run of them as they are used together.

Tolerances, fixed before the first run:
* norm: the mean of up to 16384 squares takes at most 16 + 5 + 5 roundings of 2^-24 on any path
  of the sum (a thread's own, its warp's, the block's; a warp's row: 64 + 5), half of which reaches
  y through the root, and six more follow: 41 * 2^-24 = 2.5e-6 of the value; bf16 and e4m3
  outputs add half a step, e4m3 scales the 2.5e-6 alone.  Sums and e4m3 codes: the same.
* projections: every product of two bf16 or e4m3 entries is exact; a sum of k of them is taken 16
  at a time, each step off by at most 2^-23 of the magnitudes summed so far: (k / 16 + 8) 2^-23
  of the sum of magnitudes.  The adapter's narrow sum likewise, its wide one by
  (rank_max + 8) 2^-23; the scales and the last additions are among the 8.  bf16 outputs add half
  a step.  Errors of one sign everywhere would be caught by the 2-norm: at most 1e-5 of the
  result's in f32 (a rounding of x A^T to bf16 would leave 1e-3 of the adapter's part).
* plans and slots: whole numbers, codes and scales, the same.
"""
import numpy as np
import pytest
import torch

import serve_ref as R

pytestmark = pytest.mark.gpu

I32 = torch.int32
NORM = 41 * 2.0 ** -24


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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dt="f32", std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(R.TORCH[dt])


# ---------------------------------------------------------------------------
# The residual's addition and the norm
# ---------------------------------------------------------------------------
def check_norm(x, res, gamma, rdt, out, scale, odt):
    h, y = R.norm(x, res, gamma, 1e-6, R.TORCH[rdt])
    if odt == "e4m3":
        s = y.abs().amax(-1) / 448.0
        assert ((scale.double() - s).abs() <= NORM * s).all()
        # (float64 holds the products; its quotients decide all but quotients 2^-52 beside a border)
        q = h * gamma.double()
        assert torch.equal(out.float().double(), R.e4m3(448.0 * q / q.abs().amax(-1, keepdim=True)))
    else:
        bound = NORM * y.abs() + (R.HALF["bf16"] * y.abs() * (1 + NORM) if odt == "bf16" else 0)
        assert ((out.double() - y).abs() <= bound).all()
    return h


@pytest.mark.parametrize("rows,n", [(1, 8), (3, 72), (1, 2048), (33, 1000), (700, 512), (650, 1024), (617, 1896), (609, 2048),
                                    (610, 2056), (2, 4096), (3, 5000), (2, 16384)])
@pytest.mark.parametrize("xdt,rdt,odt", [("f32", "f32", "bf16"), ("bf16", "bf16", "e4m3"), ("f32", "bf16", "f32"),
                                         ("bf16", "f32", "e4m3"), ("bf16", None, "bf16"), ("f32", None, "e4m3")])
def test_norm(tts, rows, n, xdt, rdt, odt):
    g = gen(rows * 31 + n)
    pad = 16
    x = randn(g, rows, n + pad, dt=xdt)[:, :n]
    res = None if rdt is None else (randn(g, rows, n + 2 * pad) * torch.exp(randn(g, n + 2 * pad))).to(R.TORCH[rdt])[:, :n]
    gamma = torch.rand(n, generator=g, device="cuda") + 0.5
    wide = torch.full((rows + 1, n + pad), float("nan"), device="cuda").to(R.TORCH[odt])
    raw, step = wide.view(torch.uint8).clone(), wide.element_size()
    out = wide[:rows, :n]
    total = None if rdt is None else torch.full((rows, n + pad), 7.0, device="cuda").to(R.TORCH[rdt])
    scale = torch.full((rows + 1,), 7.0, device="cuda") if odt == "e4m3" else None
    tts.tts_add_rms_norm(x, res, None if rdt is None else total[:, :n], gamma, 1e-6, out, out_scale=scale)
    h = check_norm(x, res, gamma, rdt or "f32", out, None if scale is None else scale[:rows], odt)
    if rdt is not None:
        assert torch.equal(total[:, :n].double(), h) and (total[:, n:].float() == 7.0).all()
    now = wide.view(torch.uint8)
    assert torch.equal(now[:rows, n * step:], raw[:rows, n * step:]) and torch.equal(now[rows], raw[rows])
    assert scale is None or scale[rows] == 7.0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_codes_on_the_border(tts, dt):
    """bf16 entries and a norm weight of ones: one in 200 quotients is exactly between two codes."""
    x = randn(gen(3), 400, 520, dt="bf16").to(R.TORCH[dt])
    x[:64] = torch.randint(-56, 57, (64, 520), device="cuda").to(x.dtype) / 32   # mostly ties: the largest is 56 / 32
    out, scale = torch.empty(400, 520, device="cuda", dtype=torch.float8_e4m3fn), torch.empty(400, device="cuda")
    gamma = torch.ones(520, device="cuda")
    tts.tts_add_rms_norm(x, None, None, gamma, 1e-6, out, out_scale=scale)
    check_norm(x, None, gamma, "f32", out, scale, "e4m3")


@pytest.mark.parametrize("rows", [5, 700])
def test_norm_in_place_and_without_a_stored_sum(tts, rows):
    g = gen(5)
    x, res = randn(g, rows, 264), randn(g, rows, 264)
    gamma = torch.rand(264, generator=g, device="cuda")
    a, b, s = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    tts.tts_add_rms_norm(x, res, s, gamma, 1e-5, a)
    tts.tts_add_rms_norm(x, res, None, gamma, 1e-5, b)
    assert torch.equal(a, b)
    x2, r2 = x.clone(), res.clone()
    tts.tts_add_rms_norm(x2, r2, r2, gamma, 1e-5, x2)
    assert torch.equal(r2, s) and torch.equal(x2, a)


@pytest.mark.parametrize("rows", [6, 640])
def test_norm_rows_of_zeros_infinities_and_nan_stay_alone(tts, rows):
    g = gen(6)
    x = randn(g, rows, 512)
    x[0] = 0.0
    x[1, 3] = float("inf")
    x[2, 511] = float("nan")
    gamma = torch.ones(512, device="cuda")
    out, scale = torch.empty(rows, 512, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda")
    tts.tts_add_rms_norm(x, None, None, gamma, 1e-6, out, out_scale=scale)
    assert (out[:3].view(torch.uint8) == 0).all()
    assert scale[0] == 0 and scale[1:3].isnan().all() and scale[3:].isfinite().all()
    check_norm(x[3:], None, gamma, "f32", out[3:], scale[3:], "e4m3")
    y = torch.empty_like(x)
    tts.tts_add_rms_norm(x, None, None, gamma, 1e-6, y)
    assert (y[0] == 0).all() and y[1:3].isnan().any(1).all() and y[3:].isfinite().all()


# ---------------------------------------------------------------------------
# Projections with adapters
# ---------------------------------------------------------------------------
def quantised(x):
    s = (x.abs().amax(-1) / 448.0).clamp_min(1e-12)
    return (x / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), s


def project_case(seed, rows, n, k, xdt, pool=None, rank_max=16, pad=0):
    g = gen(seed)
    c = {"x_scale": None, "w_scale": None, "a": None}
    x, w = randn(g, rows, k), randn(g, n, k, std=0.05)
    if xdt == "e4m3":
        (c["x"], c["x_scale"]), (c["w"], c["w_scale"]) = quantised(x), quantised(w)
    else:
        c["x"], c["w"] = x.bfloat16(), w.bfloat16()
    if pad:
        wide = torch.zeros(rows, k + pad, device="cuda").to(c["x"].dtype)
        wide[:, :k] = c["x"]
        c["x"] = wide[:, :k]
    if pool:
        rank = torch.randint(0, rank_max + 1, (pool,), generator=g, device="cuda", dtype=I32)
        rank[0], rank[-1] = rank_max, max(1, rank_max // 3)
        live = torch.arange(rank_max, device="cuda") < rank[:, None]
        c["rank"], c["scale"] = rank, torch.rand(pool, generator=g, device="cuda") * 2 - 0.5
        # what lies behind an adapter's rank is poison
        c["a"] = torch.where(live[..., None], randn(g, pool, rank_max, k, std=k ** -0.5), float("nan")).bfloat16()
        c["b"] = torch.where(live[:, None], randn(g, pool, n, rank_max, std=0.2), float("nan")).bfloat16()
    return c


def run_project(tts, c, adapter=None, row_stream=None, stream_adapter=None, odt="f32", pad=0, ws=None, ef=None, stream=None,
                out=None):
    rows, k = c["x"].shape
    n = c["w"].shape[0]
    if out is None:
        out = torch.full((rows, n + pad), -77.0, device="cuda").to(R.TORCH[odt])
    pool = None
    if c["a"] is not None:
        pool = tts.adapters(c["a"], c["b"], rank=c["rank"], scale=c["scale"])
        ws = tts.project_workspace(rows, n, k, c["x"].dtype, pool) if ws is None else ws
    tts.tts_project_rows(c["x"], c["w"], out[:, :n], ws, x_scale=c["x_scale"], w_scale=c["w_scale"], adapters=pool,
                         stream_adapter=adapter if stream_adapter is None else stream_adapter, row_stream=row_stream,
                         err_flag=ef, stream=stream)
    return out


def check_project(c, out, adapter, dead=None, odt="f32", norm=True):
    n, k = c["w"].shape
    rm = 0 if c["a"] is None else c["a"].shape[1]
    rows = c["x"].shape[0]
    adapter = torch.full((rows,), -1) if adapter is None else adapter.cpu()
    y, mass = R.project(c["x"], c["w"], c["a"], c.get("b"), None if c["a"] is None else c["rank"].clamp(0, rm),
                        c.get("scale"), adapter, c["x_scale"], c["w_scale"])
    live = torch.ones(rows, dtype=torch.bool, device="cuda") if dead is None else ~dead
    got = out[:, :n].double()[live]
    y, mass = y[live], mass[live]
    bound = (k / 16 + 8 + rm + 8 + k / 16 + 8) * 2.0 ** -23 * mass + 1e-30
    if odt == "bf16":
        bound = bound + R.HALF["bf16"] * y.abs() * (1 + 2.0 ** -8)
    assert torch.isfinite(got).all()
    worst = ((got - y).abs() / bound).max().item() if y.numel() else 0.0
    assert worst <= 1.0, worst
    if norm and y.numel():
        assert (got - y).norm() <= (1e-5 if odt == "f32" else 1e-2) * y.norm()
    assert (out[:, n:].float() == -77.0).all() or out.shape[1] == n
    if dead is not None:
        assert (out[dead].float() == torch.tensor(-77.0, device="cuda").to(out.dtype).float()).all()


SIZES = [(1, 1, 16), (1, 2048, 1024), (2, 7, 48), (5, 130, 64), (16, 128, 80), (17, 256, 2048), (32, 4096, 2048), (33, 200, 272),
         (64, 384, 512), (65, 129, 1024), (127, 1000, 160), (128, 2048, 256), (130, 257, 64), (256, 640, 1024), (300, 512, 2064),
         (1000, 300, 128), (1025, 1152, 4096), (2500, 264, 512)]


@pytest.mark.parametrize("rows,n,k", SIZES)
@pytest.mark.parametrize("xdt", ["bf16", "e4m3"])
def test_projection_alone(tts, rows, n, k, xdt):
    c = project_case(rows + n, rows, n, k, xdt, pad=16 if rows % 2 else 0)
    check_project(c, run_project(tts, c, pad=k % 7), None)


@pytest.mark.parametrize("rows,n,k", SIZES)
@pytest.mark.parametrize("xdt,odt,rank_max,pool", [("bf16", "f32", 16, 5), ("e4m3", "bf16", 8, 3), ("bf16", "bf16", 64, 9),
                                                   ("e4m3", "f32", 128, 4), ("bf16", "f32", 40, 70)])
def test_every_row_its_own_adapter(tts, rows, n, k, xdt, odt, rank_max, pool):
    c = project_case(rows * 3 + n + rank_max, rows, n, k, xdt, pool, rank_max)
    adapter = torch.randint(-1, pool, (rows,), generator=gen(rows), device="cuda", dtype=I32)
    ef = flag()
    check_project(c, run_project(tts, c, adapter, odt=odt, ef=ef), adapter, odt=odt)
    assert ef.item() == 0


@pytest.mark.parametrize("lengths,dead", [([300], 0), ([1, 1, 200, 3], 5), ([16, 16, 16, 16, 64, 64], 0), ([15, 17, 100, 129, 40], 1),
                                          ([700, 1, 1, 1, 500, 33], 40), ([128, 128, 256, 512], 0), ([0, 2000, 0, 30], 300),
                                          ([64] * 20, 0), ([1] * 40 + [90], 2)])
@pytest.mark.parametrize("xdt,odt,rank_max", [("bf16", "f32", 16), ("e4m3", "bf16", 64), ("bf16", "f32", 128), ("e4m3", "f32", 24)])
def test_segments_of_requests(tts, lengths, dead, xdt, odt, rank_max):
    rows, pool = sum(lengths) + dead, 6
    c = project_case(rows + rank_max, rows, 392, 320, xdt, pool, rank_max)
    of = torch.cat([torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths)), torch.full((dead,), -1)])
    sa = torch.tensor([(3 * i) % (pool + 1) - 1 for i in range(len(lengths))], dtype=I32)
    adapter = torch.where(of >= 0, sa[of.clamp(min=0)], -1)
    ef = flag()
    out = run_project(tts, c, row_stream=of.to("cuda", I32), stream_adapter=sa.cuda(), odt=odt, ef=ef)
    check_project(c, out, adapter, dead=(of < 0).cuda(), odt=odt)
    assert ef.item() == 0


# enough tiles for the pairs of SMs: lengths of the requests, rows without one, n, k
MANY = [([700], 0, 4096, 512), ([1999], 1, 2100, 272), ([160] * 6, 0, 3080, 64), ([64, 96, 160, 33, 127, 31, 1, 200, 90], 30, 3800, 80),
        ([100, 60, 150, 10, 7, 153, 300, 20, 5, 5, 5, 5, 140], 0, 4096, 336), ([1] * 170 + [2, 3, 9, 8, 7] * 20, 9, 5200, 128),
        ([31, 33] * 14, 0, 3400, 2064), ([480, 0, 0, 480], 64, 3088, 192)]


@pytest.mark.parametrize("lengths,dead,n,k", MANY)
@pytest.mark.parametrize("xdt,odt,rank_max", [("bf16", "f32", 16), ("e4m3", "bf16", 64), ("bf16", "bf16", 128), ("e4m3", "f32", 40),
                                              ("bf16", "bf16", None), ("e4m3", "f32", None)])
def test_many_rows(tts, lengths, dead, n, k, xdt, odt, rank_max):
    rows, pool = sum(lengths) + dead, 7
    c = project_case(rows + n, rows, n, k, xdt, None if rank_max is None else pool, rank_max)
    of = torch.cat([torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths)), torch.full((dead,), -1)])
    sa = torch.tensor([(3 * i) % (pool + 1) - 1 for i in range(len(lengths))], dtype=I32)
    if rank_max is None:
        sa[:] = -1
    adapter = torch.where(of >= 0, sa[of.clamp(min=0)], -1)
    ef = flag()
    out = run_project(tts, c, row_stream=of.to("cuda", I32), stream_adapter=None if rank_max is None else sa.cuda(), odt=odt, ef=ef,
                      pad=3)
    check_project(c, out, adapter, dead=(of < 0).cuda(), odt=odt)
    assert ef.item() == 0
    assert torch.equal(out, run_project(tts, c, row_stream=of.to("cuda", I32), stream_adapter=None if rank_max is None else sa.cuda(),
                                        odt=odt, pad=3))


def test_many_rows_each_its_own_adapter_and_a_bad_one(tts):
    c = project_case(33, 900, 4000, 128, "bf16", 6, 16)
    c["a"], c["b"] = c["a"].nan_to_num(0.5), c["b"].nan_to_num(0.25)
    c["rank"][:] = ints([16, 13, 7, 1, 8, 16])
    adapter = torch.randint(-1, 6, (900,), generator=gen(34), device="cuda", dtype=I32)
    check_project(c, run_project(tts, c, adapter), adapter)
    runs = torch.repeat_interleave(ints([0, 1, 2, 3, 0, 4, 5, 1]), torch.tensor([200, 100, 57, 43, 160, 40, 200, 100], device="cuda"))
    for of in (adapter, runs):
        d = dict(c, a=c["a"].clone(), b=c["b"].clone())
        d["b"][1, 5, 0] = float("inf")
        d["b"][1, 3000, 0] = float("nan")
        d["a"][4, 0, 3] = float("nan")
        got, clean = run_project(tts, d, of), run_project(tts, c, of)
        good = (of != 1) & (of != 4)
        assert torch.equal(got[good], clean[good]) and got[of == 4].isnan().all()
        one = got[of == 1]
        assert not one[:, 5].isfinite().any() and one[:, 3000].isnan().all() and (~one.isfinite()).sum() == 2 * one.shape[0]


@pytest.mark.parametrize("rows", [40, 300])
def test_requests_in_any_order_with_dead_rows_between(tts, rows):
    c = project_case(9, rows, 260, 192, "bf16", 5, 32)
    g = gen(10)
    of = torch.randint(-1, 7, (rows,), generator=g, device="cuda", dtype=I32)
    sa = ints([0, 4, -1, 2, 0, 3, 1])
    adapter = torch.where(of >= 0, sa[of.clamp(min=0).long()], -1)
    out = run_project(tts, c, row_stream=of, stream_adapter=sa)
    check_project(c, out, adapter, dead=of < 0)


@pytest.mark.parametrize("rows,lengths", [(30, None), (200, None), (600, [100, 200, 37, 263])])
@pytest.mark.parametrize("xdt", ["bf16", "e4m3"])
def test_a_bad_adapter_or_row_reaches_its_own_rows_alone(tts, rows, lengths, xdt):
    c = project_case(11, rows, 300, 128, xdt, 4, 16)
    c["rank"][:] = ints([16, 16, 13, 9])
    live = torch.arange(16, device="cuda") < c["rank"][:, None]
    g = gen(12)
    c["a"] = torch.where(live[..., None], randn(g, 4, 16, 128), float("nan")).bfloat16()
    c["b"] = torch.where(live[:, None], randn(g, 4, 300, 16), float("nan")).bfloat16()
    c["b"][1, 5, 3] = float("inf")
    c["b"][1, 7] = float("nan")
    c["a"][2, 4, 100] = float("nan")
    if lengths is None:
        adapter = ints([i % 4 for i in range(rows)])
    else:
        adapter = torch.repeat_interleave(ints([0, 1, 2, 3]), torch.tensor(lengths, device="cuda"))
    out = run_project(tts, c, adapter)[:, :300]
    good = (adapter == 0) | (adapter == 3)
    clean = dict(c, a=c["a"].nan_to_num(0.0, 0.0, 0.0), b=c["b"].nan_to_num(0.0, 0.0, 0.0))
    check_project(clean, torch.where(good[:, None], out, run_project(tts, clean, adapter)[:, :300]), adapter)
    one = adapter == 1
    assert not out[one][:, 5].isfinite().any() and out[one][:, 7].isnan().all()
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[5] = keep[7] = False
    assert out[one][:, keep].isfinite().all()
    assert out[adapter == 2].isnan().all()
    # a row
    c = project_case(13, rows, 300, 128, xdt, 4, 16)
    if xdt == "bf16":
        c["x"][3, 17] = float("nan")
    else:
        c["x_scale"][3] = float("nan")
    out = run_project(tts, c, adapter)[:, :300]
    assert out[3].isnan().all() and out[:3].isfinite().all() and out[4:].isfinite().all()


def test_ids_and_ranks_out_of_range(tts):
    c = project_case(14, 6, 64, 64, "bf16", 3, 16)
    c["rank"] = ints([16, -4, 99])
    g = gen(15)
    c["a"], c["b"] = randn(g, 3, 16, 64, dt="bf16", std=0.1), randn(g, 3, 64, 16, dt="bf16")
    for of, sa, want, bits_ in (([0, 1, 2, 3, 9, -5], [0, 3, -1, 0], [0, -1, -1, 0, -1, -1], tts.EFLAG_ID_RANGE),
                                ([0, 0, 1, 1, 1, 0], [1, 2], [1, 1, 2, 2, 2, 1], tts.EFLAG_NVALID)):
        ef = flag()
        out = run_project(tts, c, row_stream=ints(of), stream_adapter=ints(sa), ef=ef)
        assert ef.item() == bits_
        check_project(c, out, torch.tensor(want), dead=ints(of) < 0)


def test_an_adapter_beside_no_shared_weights_is_held_in_32_bits(tts):
    # W = 0: the output is the adapter's part alone, so its 2-norm shows how x A^T was held
    for rows in (20, 400):
        for odt in ("f32", "bf16"):
            c = project_case(16, rows, 256, 512, "bf16", 2, 64)
            c["w"].zero_()
            c["rank"][:] = 64
            g = gen(17)
            c["a"], c["b"] = randn(g, 2, 64, 512, dt="bf16", std=0.05), randn(g, 2, 256, 64, dt="bf16")
            adapter = (torch.arange(rows, device="cuda") >= rows // 2).to(I32)
            out = run_project(tts, c, adapter, odt=odt)
            y, _ = R.project(c["x"], c["w"], c["a"], c["b"], c["rank"], c["scale"], adapter.cpu())
            assert (out.double() - y).norm() <= (1e-6 if odt == "f32" else 2.0 ** -9) * y.norm()


def test_a_workspace_is_enough_for_fewer_rows_and_holds_nothing(tts):
    c = project_case(18, 500, 256, 256, "bf16", 4, 32)
    adapter = torch.randint(-1, 4, (500,), generator=gen(19), device="cuda", dtype=I32)
    pool = tts.adapters(c["a"], c["b"], rank=c["rank"], scale=c["scale"])
    ws = tts.project_workspace(500, 256, 256, "bf16", pool)
    ws.fill_(255)   # NaN everywhere
    first = run_project(tts, c, adapter, ws=ws)
    check_project(c, first, adapter)
    for rows in (1, 33, 100, 257, 499):
        d = dict(c, x=c["x"][:rows])
        ws.fill_(255)
        check_project(d, run_project(tts, d, adapter[:rows].contiguous(), ws=ws), adapter[:rows])
    assert torch.equal(run_project(tts, c, adapter, ws=ws), first)


@pytest.mark.parametrize("rows,n", [(1, 520), (32, 520), (100, 520), (700, 520), (1000, 3100)])
@pytest.mark.parametrize("xdt", ["bf16", "e4m3"])
def test_projection_replayed_and_on_two_streams(tts, rows, n, xdt):
    c = project_case(20, rows, n, 1024, xdt, 4, 32)
    adapter = torch.randint(-1, 4, (rows,), generator=gen(21), device="cuda", dtype=I32)
    eager = run_project(tts, c, adapter)
    check_project(c, eager, adapter)
    pool = tts.adapters(c["a"], c["b"], rank=c["rank"], scale=c["scale"])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [tts.project_workspace(rows, n, 1024, xdt, pool) for _ in streams]
    outs = [torch.zeros_like(eager) for _ in streams]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=streams[0]):
        run_project(tts, c, adapter, ws=spaces[0], out=outs[0], stream=streams[0])
    for _ in range(3):
        outs[0].fill_(-77.0)
        outs[1].fill_(-77.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            for _ in range(4):
                run_project(tts, c, adapter, ws=spaces[1], out=outs[1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager)
    # another batch in the same graph: the device data decide
    adapter.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    check_project(c, outs[0], adapter)


# ---------------------------------------------------------------------------
# Pages and row maps
# ---------------------------------------------------------------------------
class Pool:
    """A paged cache's table and list, with maps, on the device and as the restatement sees them."""

    def __init__(self, tts, B, capacity, page, n_pages, max_rows, T=0, seed=0, extra=0):
        g = torch.Generator().manual_seed(seed)
        self.tts, self.B, self.capacity, self.page, self.n_pages, self.T = tts, B, capacity, page, n_pages, T
        self.max_rows = B * T if T else max_rows
        self.table = torch.full((B, capacity // page + extra), -1, dtype=I32, device="cuda")
        if extra:
            self.table[:, capacity // page:] = 12345
        self.free = torch.randperm(n_pages, generator=g).to("cuda", I32)
        self.n_free = ints([n_pages])
        self.desc = tts.kv_desc(B, 16, 8, 128, capacity, "bf16", window_quantum=1, paged=True, page_size=page, n_pages=n_pages,
                                block_table=self.table)
        self.extra = extra
        z = lambda n, dt=I32: torch.full((n,), 55, dtype=dt, device="cuda")  # noqa: E731
        self.n_rows, self.row_start = z(B), z(B + 1)
        self.row_stream, self.row_pos, self.row_slot = z(self.max_rows), z(self.max_rows), z(self.max_rows, torch.int64)

    def call(self, past, new, ef=None):
        self.tts.tts_page_plan(self.desc, self.table, self.free, self.n_free, past, new, self.n_rows, self.row_start,
                               self.row_stream, self.row_pos, self.row_slot, T=self.T, err_flag=ef)

    def step(self, past, new):
        per = self.capacity // self.page
        want = R.plan(self.table[:, :per].tolist(), self.free.tolist(), int(self.n_free), past, new, self.n_pages, self.page,
                      self.capacity, self.max_rows, self.T)
        ef = flag()
        self.call(ints(past), ints(new), ef)
        assert (self.table[:, :per].cpu().numpy() == want["table"]).all()
        assert (self.table[:, per:] == 12345).all()
        assert (self.free.cpu().numpy() == want["free"]).all() and int(self.n_free) == want["n_free"]
        for key in ("n_rows", "row_start", "row_stream", "row_pos", "row_slot"):
            assert getattr(self, key).tolist() == want[key], key
        bits_ = {"page": self.tts.EFLAG_PAGE, "nvalid": self.tts.EFLAG_NVALID}
        assert ef.item() == sum(bits_[f] for f in want["flags"])
        return want


@pytest.mark.parametrize("B,capacity,page,n_pages,max_rows,T", [
    (1, 1, 1, 1, 1, 0), (1, 64, 16, 4, 64, 0), (3, 64, 8, 20, 40, 0), (5, 256, 256, 7, 300, 0), (64, 512, 16, 1500, 700, 0),
    (130, 96, 1, 9000, 3000, 0), (700, 128, 16, 3000, 9000, 0), (4096, 64, 16, 9000, 30000, 0), (4, 64, 16, 16, 0, 7),
    (40, 256, 64, 100, 0, 64), (600, 512, 16, 9000, 0, 40), (2, 32768, 16, 4096, 40000, 0), (17, 320, 32, 90, 100, 0)])
def test_plans_step_by_step(tts, B, capacity, page, n_pages, max_rows, T):
    rng = np.random.RandomState(B * 7 + page)
    pool = Pool(tts, B, capacity, page, n_pages, max_rows, T, seed=B, extra=B % 3)
    past = [0] * B
    top = T or max(1, min(capacity, (2 * pool.max_rows) // B))
    for step in range(6):
        kind = rng.rand(B)
        new = np.where(kind < 0.15, -1, np.where(kind < 0.3, 0, np.where(kind < 0.7, 1, rng.randint(1, top + 1, B))))
        new = [int(x) for x in new]
        if step == 4:   # what a caller gets wrong
            new[rng.randint(B)] = capacity + 1
            past_ = list(past)
            past_[rng.randint(B)] = -1
            want = pool.step(past_, new)
            continue
        new = [min(n, max(0, capacity - p)) if n > 0 else n for n, p in zip(new, past)]
        want = pool.step(past, new)
        # a drafted step keeps a part of its rows only; the pages stay
        past = [0 if n < 0 else p + (rng.randint(1, r + 1) if r and step % 2 else r) for p, n, r in zip(past, new, want["n_rows"])]


def test_plan_pages_run_out_and_come_back(tts):
    pool = Pool(tts, 4, 64, 16, 5, 200)
    w = pool.step([0, 0, 0, 0], [33, 20, 17, 1])     # 3 + 2 pages, then none
    assert w["n_rows"] == [33, 20, 0, 0]
    w = pool.step([33, 20, 0, 0], [1, 1, 1, 1])      # those with room in their pages go on
    assert w["n_rows"] == [1, 1, 0, 0]
    w = pool.step([34, 21, 0, 0], [-1, 1, 40, 1])    # the pages of an ended stream serve the same step
    assert w["n_rows"] == [0, 1, 40, 0] and w["n_free"] == 0
    w = pool.step([0, 22, 40, 0], [-1, -1, -1, -1])
    assert w["n_free"] == 5 and sorted(pool.free.tolist()) == [0, 1, 2, 3, 4]
    w = pool.step([0] * 4, [-1] * 4)                 # ended twice: nothing to return
    assert w["n_free"] == 5


def test_plan_rows_that_do_not_fit(tts):
    pool = Pool(tts, 5, 64, 16, 40, 50)
    w = pool.step([0] * 5, [20, 30, 1, 0, 2])
    assert w["n_rows"] == [20, 30, 0, 0, 0] and w["flags"] == {"nvalid"}
    pool = Pool(tts, 3, 2 ** 20, 256, 5000, 100)
    w = pool.step([0] * 3, [2 ** 20, 2 ** 20, 7])    # sums far over max_rows
    assert w["n_rows"] == [0, 0, 0]


def test_plan_with_a_damaged_list(tts):
    pool = Pool(tts, 2, 64, 16, 6, 64)
    pool.n_free.fill_(9)                             # more than the list holds
    pool.free[5] = 77                                # a page that does not exist
    w = pool.step([0, 0], [20, 3])
    assert w["flags"] == {"nvalid", "page"} and -1 in w["row_slot"][:20]
    pool.table[1] = ints([0, 1, 2, 3])               # held twice: the list cannot take them all
    w = pool.step([0, 0], [0, -1])
    assert w["n_free"] <= 6
    pool.n_free.fill_(-3)
    pool.step([0, 0], [0, 1])


def test_plan_arrays_may_begin_at_any_entry(tts):
    pool = Pool(tts, 5, 64, 16, 20, 40)
    for key in ("free", "n_free", "n_rows", "row_start", "row_stream", "row_pos", "row_slot"):
        t = getattr(pool, key)
        setattr(pool, key, torch.cat([t[:1], t])[1:])
    call = pool.call
    pool.call = lambda past, new, ef: call(torch.cat([past[:1], past])[1:], torch.cat([new[:1], new])[1:], ef)
    pool.step([0] * 5, [17, 1, 0, -1, 20])
    pool.step([17, 1, 0, 0, 20], [-1, 16, 3, 5, 1])


@pytest.mark.parametrize("max_rows", [900, 20000])
def test_plan_replayed(tts, max_rows):
    a, b = (Pool(tts, 40, 512, 16, 2000, max_rows, seed=3) for _ in range(2))
    past, new = ints([0] * 40), ints([0] * 40)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        a.call(past, new)
    rng = np.random.RandomState(4)
    p = [0] * 40
    for step in range(5):
        n = [int(x) for x in rng.choice([-1, 0, 1, 25], 40)]
        past.copy_(ints(p))
        new.copy_(ints(n))
        graph.replay()
        w = b.step(p, n)
        for key in ("table", "free", "n_free", "n_rows", "row_start", "row_stream", "row_pos", "row_slot"):
            assert torch.equal(getattr(a, key), getattr(b, key)), key
        p = [0 if x < 0 else q + r for x, q, r in zip(n, p, w["n_rows"])]


# ---------------------------------------------------------------------------
# Rows by slot
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,hkv,d,page,src,kv", [
    (1, 8, 128, 16, "f32", "bf16"), (7, 1, 64, 1, "bf16", "f32"), (40, 5, 64, 8, "f32", "i8"), (100, 8, 128, 256, "bf16", "e4m3"),
    (33, 3, 128, 0, "bf16", "bf16"), (300, 2, 64, 16, "f32", "e4m3"), (64, 8, 128, 0, "f32", "i8"), (9, 7, 128, 32, "f32", "f32")])
def test_slots_write_what_positions_write(tts, rows, hkv, d, page, src, kv):
    g = gen(rows + d)
    size = page or 64
    n_pages = rows // size + 4
    dt = R.TORCH[kv]
    caches = []
    for _ in range(2):
        raw = [torch.full((n_pages, hkv, size, d), 3, dtype=torch.uint8, device="cuda").view(dt) if dt.itemsize == 1
               else torch.full((n_pages, hkv, size, d), 3.0, dtype=dt, device="cuda") for _ in range(2)]
        sc = [torch.full((n_pages, hkv, size), 9.0, device="cuda") for _ in range(2)] if dt.itemsize == 1 else []
        caches.append((raw + sc, tts.kv_cache(*raw, *sc)))
    x = (randn(g, rows, 2 * hkv * d + 16) * torch.exp(2 * randn(g, rows, 1))).to(R.TORCH[src])
    x[0, :d] = 0.0
    if rows > 5:
        x[5, 3] = float("nan")
        x[4, hkv * d] = float("inf")
    slots = torch.randperm(n_pages * size, generator=g, device="cuda")[:rows].to(torch.int64)
    skip = torch.zeros(rows, dtype=torch.bool, device="cuda")
    skip[2::6] = True
    desc = tts.kv_desc(1 if page else n_pages, hkv, hkv, d, size, kv, window_quantum=1, paged=page > 0, page_size=page,
                       n_pages=n_pages, block_table=ints([[0]]) if page else None)
    ef = flag()
    tts.tts_kv_write_slots(x[:, :hkv * d], x[:, hkv * d:2 * hkv * d], caches[0][1], desc, torch.where(skip, -1 - slots, slots),
                           err_flag=ef)
    assert ef.item() == 0
    # the same rows, one a stream, through a table that names each row's page (a contiguous cache
    # is a pool of pages as long as its streams)
    y, at = x[~skip].contiguous(), slots[~skip]
    table = (at // size).to(I32)[:, None].contiguous()
    one = tts.kv_desc(at.numel(), hkv, hkv, d, size, kv, window_quantum=1, paged=True, page_size=size, n_pages=n_pages,
                      block_table=table)
    tts.tts_kv_write_rows(y[:, :hkv * d], y[:, hkv * d:2 * hkv * d], caches[1][1], one, (at % size).to(I32), 1)
    for a, e in zip(caches[0][0], caches[1][0]):
        assert torch.equal(a.view(torch.uint8), e.view(torch.uint8))


def test_slots_past_the_end_are_skipped(tts):
    k = torch.ones(4, 128, device="cuda")
    raw = [torch.zeros(3, 2, 8, 64, device="cuda") for _ in range(2)]
    desc = tts.kv_desc(3, 2, 2, 64, 8, "f32", window_quantum=1)
    ef = flag()
    slot = torch.tensor([24, 23, 2 ** 40, -2 ** 60], device="cuda")
    tts.tts_kv_write_slots(k, k, tts.kv_cache(*raw), desc, slot, err_flag=ef)
    assert ef.item() == tts.EFLAG_POS_RANGE
    for t in raw:
        assert (t[2, :, 7] == 1).all() and t.sum() == 128


# ---------------------------------------------------------------------------
# Together: steps of requests that come and go
# ---------------------------------------------------------------------------
def serve_steps(tts, dev, T, kv, xdt, captured):
    """Four steps of six requests, one layer's front half: plan, norm, projection with adapters,
    rotary rows, cache rows by slot, attention of the step's rows.  Returns what each step's live
    rows attended to, with the inputs, for a dense 64-bit restatement."""
    B, hid, hq, hkv, d, page, cap = 6, 256, 4, 2, 64, 8, 64
    n = (hq + 2 * hkv) * d
    rows = B * T
    g = gen(50 + T)
    w, pool_a, pool_b = randn(g, n, hid, std=0.1), randn(g, 3, 16, hid, dt="bf16", std=0.05), randn(g, 3, n, 16, dt="bf16", std=0.2)
    wq, ws_ = quantised(w) if xdt == "e4m3" else (w.bfloat16(), None)
    gamma, gq = torch.rand(hid, generator=g, device=dev) + 0.5, torch.rand(d, generator=g, device=dev) + 0.5
    rank, scale, sa = ints([16, 5, 12]), torch.tensor([1.0, -0.5, 2.0], device=dev), ints([0, 2, -1, 1, 1, 0])
    pool = Pool(tts, B, cap, page, 40, 0, T, seed=8)
    dt = R.TORCH[kv]
    raw = [torch.zeros(40, hkv, page, d, device=dev).to(dt) for _ in range(2)]
    sc = [torch.zeros(40, hkv, page, device=dev) for _ in range(2)] if dt.itemsize == 1 else [None, None]
    cache = tts.kv_cache(*raw, *sc)
    desc = tts.kv_desc(B, hq, hkv, d, cap, kv, window_quantum=8, paged=True, page_size=page, n_pages=40, block_table=pool.table)
    cs = torch.empty(cap, d // 2, 2, device=dev)
    tts.tts_rope_table(cs, cap, d, 1e4)
    ad = tts.adapters(pool_a, pool_b, rank=rank, scale=scale)
    pws = tts.project_workspace(rows, n, hid, xdt, ad)
    tws = tts.tree_workspace(desc, T, "bf16")
    x, res = torch.zeros(rows, hid, device=dev), torch.zeros(rows, hid, device=dev)
    h = torch.zeros(rows, hid, device=dev)
    hq8 = torch.zeros(rows, hid, device=dev).to(wq.dtype)
    hs = torch.zeros(rows, device=dev) if xdt == "e4m3" else None
    qkv = torch.zeros(rows, n, device=dev)
    q, k = torch.zeros(rows, hq * d, dtype=torch.bfloat16, device=dev), torch.zeros(rows, hkv * d, dtype=torch.bfloat16, device=dev)
    v = torch.zeros(rows, hkv * d, dtype=torch.bfloat16, device=dev)
    out = torch.zeros(B, T, hq, d, dtype=torch.bfloat16, device=dev)
    past, new, ef = ints([0] * B), ints([0] * B), flag()

    def step():
        pool.call(past, new, ef)
        tts.tts_add_rms_norm(x, res, h, gamma, 1e-6, hq8, out_scale=hs)
        tts.tts_project_rows(hq8, wq, qkv, pws, x_scale=hs, w_scale=ws_, adapters=ad, stream_adapter=sa,
                             row_stream=pool.row_stream, err_flag=ef)
        tts.tts_rope_rows(qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], q, k, pool.row_pos, hq, hkv, d, cs, gamma_q=gq, gamma_k=gq)
        v.copy_(qkv[:, (hq + hkv) * d:])
        tts.tts_kv_write_slots(k, v, cache, desc, pool.row_slot, err_flag=ef)
        tts.tts_tree_attn(q, cache, desc, past, T, d ** -0.5, out, tws, n_nodes=pool.n_rows, err_flag=ef)

    graph = None
    if captured:
        step()   # (nothing is asked for yet: no stream has rows)
        stream = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            step()
    rng = np.random.RandomState(9)
    p, seen = [0] * B, []
    for i in range(5):
        ask = [int(a) for a in rng.randint(1, T + 1, B)]
        ask[i] = -1 if i else ask[i]
        ask[(i + 3) % B] = 0
        x.copy_(randn(g, rows, hid))
        res.copy_(randn(g, rows, hid))
        past.copy_(ints(p))
        new.copy_(ints(ask))
        graph.replay() if captured else step()
        assert ef.item() == 0
        seen.append({"past": p, "ask": ask, "n_rows": pool.n_rows.tolist(), "x": x.clone(), "res": res.clone(), "out": out.clone(),
                     "hs": None if hs is None else hs.clone(), "hq": hq8.clone(), "q": q.clone(), "k": k.clone(), "v": v.clone(),
                     "qkv": qkv.clone()})
        p = [0 if a < 0 else b + r for a, b, r in zip(ask, p, seen[-1]["n_rows"])]
    return seen, dict(w=wq, w_scale=ws_, a=pool_a, b=pool_b, rank=rank, scale=scale, sa=sa, gamma=gamma, gq=gq, hq=hq, hkv=hkv, d=d,
                      T=T, B=B)


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("xdt", ["bf16", "e4m3"])
def test_steps_of_requests_that_come_and_go(tts, cuda_dev, T, kv, xdt):
    seen, m = serve_steps(tts, cuda_dev, T, kv, xdt, captured=False)
    again, _ = serve_steps(tts, cuda_dev, T, kv, xdt, captured=True)
    B, hq, hkv, d = m["B"], m["hq"], m["hkv"], m["d"]
    kept = [([], []) for _ in range(B)]     # each request's K and V rows, as a dense cache
    for s, t in zip(seen, again):
        live = torch.tensor([i % T < s["n_rows"][i // T] for i in range(B * T)], device="cuda")
        assert s["n_rows"] == [max(a, 0) for a in s["ask"]]
        for key in ("q", "k", "v", "qkv"):
            assert torch.equal(s[key][live], t[key][live]), key
        check_norm(s["x"], s["res"], m["gamma"], "f32", s["hq"], s["hs"], xdt)
        adapter = torch.tensor([int(m["sa"][i // T]) for i in range(B * T)])
        c = dict(m, x=s["hq"], x_scale=s["hs"])
        check_project(dict(c, x=s["hq"][live], x_scale=None if s["hs"] is None else s["hs"][live]), s["qkv"][live], adapter[live.cpu()])
        for b in range(B):
            if s["ask"][b] < 0:
                kept[b] = ([], [])
            for i in range(s["n_rows"][b]):
                for rows, key in zip(kept[b], ("k", "v")):
                    y = s[key][b * T + i].double().view(hkv, d)
                    if kv == "e4m3":
                        z = y.abs().amax(-1, keepdim=True).float() * torch.tensor(1 / 448, device="cuda")
                        y = R.e4m3(y / z.double()) * z.double()
                    rows.append(y)
            n = s["n_rows"][b]
            if n == 0:
                continue
            K, V = (torch.stack(r) for r in kept[b])
            for i in range(n):
                pos = s["past"][b] + i + 1
                for j in range(hq):
                    g = j // (hq // hkv)
                    p = torch.softmax(K[:pos, g] @ s["q"][b * T + i].double().view(hq, d)[j] * d ** -0.5, 0)
                    ref, mean = p @ V[:pos, g], p @ V[:pos, g].abs()
                    got = s["out"][b, i, j].double()
                    # the output's half step, the weights' half step and the f32 terms
                    assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -8 * mean + 2e-5 * mean.max()).all()
                    assert torch.equal(s["out"][b, i, j], t["out"][b, i, j])
