"""Inputs of the calls that serve many requests at once that the contract allows and that are easily
missed: adapters named by any negative number, infinities, terms that cancel, on each of the
projection's kernels; tables that hold more pages than there are.

Tolerances are those of test_serve_gpu (check_project); what is compared with equality is exact
in f32.
"""
import pytest
import torch

import serve_ref as R
from test_serve_gpu import I32, Pool, check_project, flag, gen, ints, project_case, randn, run_project, tts  # noqa: F401

pytestmark = pytest.mark.gpu

# Sizes that reach each of the projection's kernels: (rows, n, k, requests).  Few rows on the CUDA
# cores' adapters; rows of requests that share blocks of 16, split over a cluster; the same on
# pairs of SMs (see project_is_many).
PATHS = {"few": (40, 260, 192, 40), "blocks": (400, 300, 272, 7), "pairs": (1100, 3400, 128, 9)}


def segments(path):
    """row_stream: requests of ragged lengths, in order, and three rows of no request."""
    rows, _, _, streams = PATHS[path]
    live = rows - 3
    of = torch.arange(live) * streams // live if streams < live else torch.arange(live)
    cut = torch.tensor([(i * 5) % 11 - 5 for i in range(live)])
    return torch.cat([(of + (cut > 4)).clamp(max=streams - 1).sort().values, torch.full((3,), -1)]).to("cuda", I32)


@pytest.mark.parametrize("path", list(PATHS))
@pytest.mark.parametrize("xdt,odt", [("bf16", "f32"), ("e4m3", "bf16")])
def test_any_negative_adapter_is_the_shared_projection_alone(tts, path, xdt, odt):  # noqa: F811
    rows, n, k, streams = PATHS[path]
    c = project_case(rows, rows, n, k, xdt, 4, 16)
    of = segments(path)
    names = [-2, 1, -1, -3, 0, -2 ** 31, 3, 2, -2]
    sa = ints([names[i % len(names)] for i in range(streams)])
    adapter = torch.where(of >= 0, sa[of.clamp(min=0).long()], -1).clamp(min=-1)
    ef = flag()
    out = run_project(tts, c, row_stream=of, stream_adapter=sa, odt=odt, ef=ef, pad=3)
    check_project(c, out, adapter, dead=of < 0, odt=odt)
    assert ef.item() == 0


@pytest.mark.parametrize("path", list(PATHS))
@pytest.mark.parametrize("xdt", ["bf16", "e4m3"])
@pytest.mark.parametrize("odt", ["f32", "bf16"])
def test_narrow_products_that_cancel_keep_their_last_bits(tts, path, xdt, odt):  # noqa: F811
    """W = 0, v = t (1 + 2^-9 + 2^-18, 1 + 2^-9), B = (c, -c): out = t c 2^-18 for powers of two t and
    c, each sum on the way exact in f32.  With 16 bits of v it is 0."""
    rows, n, k, streams = PATHS[path]
    c = project_case(7, rows, n, k, xdt, 4, 16)
    t = torch.exp2((torch.arange(rows, device="cuda") % 5 - 2).float()) * (1 - torch.arange(rows, device="cuda") % 3 % 2 * 2)
    x = torch.zeros(rows, k, device="cuda")
    x[:, :3] = 1.0 if xdt == "e4m3" else t[:, None]
    c["x"] = x.to(c["x"].dtype)
    if xdt == "e4m3":
        c["x_scale"] = t.clone()
    c["w"].zero_()
    c["rank"][:] = 2
    c["scale"][:] = torch.tensor([1.0, -2.0, 0.5, 4.0], device="cuda")
    c["a"].fill_(float("nan"))
    c["b"].fill_(float("nan"))
    c["a"][:, :2] = 0.0
    c["a"][:, :2, 0], c["a"][:, :2, 1], c["a"][:, 0, 2] = 1.0, 2.0 ** -9, 2.0 ** -18
    col = torch.exp2((torch.arange(n, device="cuda") % 7 - 3).float())
    c["b"][:, :, 0], c["b"][:, :, 1] = col, -col
    of = segments(path)
    sa = ints([(3 * i) % 5 - 1 for i in range(streams)])
    adapter = torch.where(of >= 0, sa[of.clamp(min=0).long()], -1)
    out = run_project(tts, c, row_stream=of, stream_adapter=sa, odt=odt)
    want = torch.where(adapter >= 0, c["scale"][adapter.clamp(min=0).long()], 0.0)[:, None] * t[:, None] * col * 2.0 ** -18
    assert torch.equal(out[of >= 0].double(), want[of >= 0].double())


def close(out, y, mass, k, rank_max, odt):
    """Within check_project's bound of the float64 values."""
    bound = (k / 8 + rank_max + 24) * 2.0 ** -23 * mass + 1e-30
    if odt == "bf16":
        bound = bound + R.HALF["bf16"] * y.abs() * (1 + 2.0 ** -8)
    return ((out.double() - y).abs() <= bound).all()


@pytest.mark.parametrize("path", list(PATHS))
@pytest.mark.parametrize("xdt,odt", [("bf16", "f32"), ("e4m3", "bf16")])
def test_infinities_of_an_adapter_are_those_of_the_formula(tts, path, xdt, odt):  # noqa: F811
    """x A^T of small whole numbers (few bits each) against infinite entries of B of either sign, and
    an infinite scale: an infinity of the products' sign where all agree, NaN where they do not or
    where 0 meets an infinity."""
    rows, n, k, streams = PATHS[path]
    c = project_case(rows + 1, rows, n, k, xdt, 4, 16)
    g = gen(rows)
    whole = lambda *s: torch.randint(-1, 2, s, generator=g, device="cuda").float()  # noqa: E731
    c["x"] = whole(rows, k).to(c["x"].dtype)
    if xdt == "e4m3":
        c["x_scale"].fill_(1.0)
    c["rank"][:] = ints([16, 13, 1, 9])
    c["scale"][:] = torch.tensor([1.0, 0.5, float("inf"), -1.0], device="cuda")
    live = torch.arange(16, device="cuda") < c["rank"][:, None]
    c["a"] = torch.where(live[..., None], whole(4, 16, k), float("nan")).bfloat16()
    b = randn(g, 4, n, 16, dt="bf16", std=0.2).float()
    b[0, 5, 3], b[0, 6, 2], b[0, 6, 7] = float("inf"), float("inf"), float("-inf")
    b[1, 7], b[2, 9, 0], b[3, n - 1, 8] = float("inf"), float("-inf"), float("-inf")
    c["b"] = torch.where(live[:, None], b, float("nan")).bfloat16()
    of = segments(path)
    sa = ints([(3 * i) % 5 - 1 for i in range(streams)])
    adapter = torch.where(of >= 0, sa[of.clamp(min=0).long()], -1)
    out = run_project(tts, c, row_stream=of, stream_adapter=sa, odt=odt)
    for i in range(4):
        at = (adapter == i).nonzero()[:, 0]
        r = int(c["rank"][i])
        bi = c["b"][i, :, :r].double()
        v = (c["x"][at].double() @ c["a"][i, :r].double().T) * c["scale"][i].double()
        odd = (~bi.isfinite()).any(1) if i != 2 else torch.ones(n, dtype=torch.bool, device="cuda")
        assert at.numel() > 0 and odd.any()
        for col in odd.nonzero()[:, 0].tolist():
            want = (v * bi[col]).sum(1)     # (elementwise: an infinity for each that the formula has)
            got = out[at, col].double()
            assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isposinf(), want.isposinf())
            assert torch.equal(got.isneginf(), want.isneginf())
        if i != 2:
            d = dict(c, x=c["x"][at][:, :], b=c["b"].float().nan_to_num(0.0, 0.0, 0.0).bfloat16())
            y, mass = R.project(d["x"], d["w"], d["a"], d["b"], d["rank"], d["scale"], torch.full((at.numel(),), i),
                                None if xdt == "bf16" else c["x_scale"][at], c["w_scale"])
            assert close(out[at][:, ~odd], y[:, ~odd], mass[:, ~odd], k, 16, odt)


@pytest.mark.parametrize("path", list(PATHS))
@pytest.mark.parametrize("xdt,odt", [("bf16", "f32"), ("e4m3", "bf16")])
def test_narrow_products_near_the_largest_f32_stay_finite(tts, path, xdt, odt):  # noqa: F811
    """x A^T of 3.4e38, past bf16's largest value, against a small B."""
    rows, n, k, streams = PATHS[path]
    c = project_case(rows + 2, rows, n, k, xdt, 4, 16)
    x = torch.zeros(rows, k, device="cuda")
    x[:, 0] = 1 - 2 * (torch.arange(rows, device="cuda") % 2)
    c["x"] = x.to(c["x"].dtype)
    if xdt == "e4m3":
        c["x_scale"].fill_(1.0)
    c["w"].zero_()
    c["rank"][:] = 3
    c["scale"][:] = torch.tensor([3.4e38, -3.4e38, 3.4028234e38, 3.39e38], device="cuda")
    c["a"].zero_()
    c["a"][:, :3, 0] = 1.0
    c["b"] = (randn(gen(3), 4, n, 16) * 2.0 ** -120).bfloat16()
    of = segments(path)
    sa = ints([(3 * i) % 5 - 1 for i in range(streams)])
    adapter = torch.where(of >= 0, sa[of.clamp(min=0).long()], -1)
    out = run_project(tts, c, row_stream=of, stream_adapter=sa, odt=odt)
    y, mass = R.project(c["x"], c["w"], c["a"], c["b"], c["rank"], c["scale"], adapter.cpu(), c["x_scale"], c["w_scale"])
    assert close(out[of >= 0], y[of >= 0], mass[of >= 0], k, 16, odt)


@pytest.mark.parametrize("B,n_pages,listed,ended", [
    (2, 6, 0, [0, 1]),                # the second's pages begin on the list and end past it
    (3, 6, 2, [0, 1, 2]),
    (9, 5, 0, [1, 4, 8]),             # the sum is past all pages before the last
    (70, 20, 7, list(range(0, 70, 2))),
    (1100, 3000, 0, list(range(1100))),   # in the third batch of streams
    (4096, 700, 100, list(range(5, 4096)))])
def test_pages_held_twice_go_to_the_list_in_order_until_it_is_full(tts, B, n_pages, listed, ended):  # noqa: F811
    pool = Pool(tts, B, 64, 16, n_pages, 64, seed=B)
    pool.n_free.fill_(listed)
    pool.table.copy_(torch.randint(-1, n_pages, (B, 4), generator=gen(B), device="cuda", dtype=I32))
    pool.table[:2] = ints([[0, 1, 2, 3], [4, 3, 2, 1]])
    new = [-1 if b in set(ended) else 0 for b in range(B)]
    want = pool.step([0] * B, new)    # (compares table, list, maps and flags with the restatement)
    assert want["n_free"] == n_pages and want["flags"] == {"page"}
    pool.step([0] * B, [1 if n else 0 for n in new])


@pytest.mark.parametrize("xdt", ["f32", "bf16"])
def test_norm_codes_of_rows_past_the_largest_f32(tts, xdt):  # noqa: F811
    """max |y| past f32's range is an infinity in y: scale NaN, codes 0; below it the scale is finite."""
    n, rows = 512, 6
    x = randn(gen(1), rows, n).sign().to(R.TORCH[xdt]) * 1.5      # the mean square is 2.25: y = +-gamma
    gamma = torch.full((n,), 1e-3, device="cuda")
    x[1, 7] = 1.9375                   # r is just below 1 / 1.5: y = 1.29 gamma there
    x[3, 7], x[4, 7] = 1.9375, -1.9375
    gamma[7] = 3e38
    x[0, 7], x[2, 7], x[5, 7] = 1.5, 0.5, 0.0
    out, scale = torch.ones(rows, n, device="cuda").to(R.TORCH["e4m3"]), torch.empty(rows, device="cuda")
    tts.tts_add_rms_norm(x, None, None, gamma, 0.0, out, out_scale=scale)
    past = torch.tensor([False, True, False, True, True, False], device="cuda")
    y = R.norm(x, None, gamma, 0.0, None)[1].abs().amax(-1)
    assert torch.equal(y > 3.41e38, past) and (y[~past] < 3.1e38).all()
    assert torch.equal(scale.isnan(), past) and scale[~past].isfinite().all()
    assert (out[past].view(torch.uint8) == 0).all()
    assert ((scale[~past].double() - y[~past] / 448).abs() <= 41 * 2.0 ** -24 * y[~past] / 448).all()


# ---------------------------------------------------------------------------
# Requests of many rows each: what reaches the adapters' products on the tensor cores
# ---------------------------------------------------------------------------
def batch(path, xdt, seed):
    """A case with its row map and the requests' adapters, four of them and none."""
    rows, n, k, streams = PATHS[path]
    c = project_case(seed + rows, rows, n, k, xdt, 4, 32)
    c["rank"][:] = ints([32, 29, 8, 17])
    live = torch.arange(32, device="cuda") < c["rank"][:, None]
    g = gen(seed)
    c["a"] = torch.where(live[..., None], randn(g, 4, 32, k, std=k ** -0.5), float("nan")).bfloat16()
    c["b"] = torch.where(live[:, None], randn(g, 4, n, 32, std=0.2), float("nan")).bfloat16()
    of = segments(path)
    sa = ints([(3 * i) % 5 - 1 for i in range(streams)])
    return c, of, sa, torch.where(of >= 0, sa[of.clamp(min=0).long()], -1)


@pytest.mark.parametrize("path", list(PATHS))
@pytest.mark.parametrize("xdt,odt", [("bf16", "f32"), ("e4m3", "bf16")])
def test_a_bad_adapter_or_row_changes_no_other_row(tts, path, xdt, odt):  # noqa: F811
    c, of, sa, adapter = batch(path, xdt, 40)
    n = c["w"].shape[0]
    clean = run_project(tts, c, row_stream=of, stream_adapter=sa, odt=odt)
    check_project(c, clean, adapter, dead=of < 0, odt=odt)
    d = dict(c, a=c["a"].clone(), b=c["b"].clone())
    d["b"][1, 5, 3], d["b"][1, 7], d["b"][1, n - 1, 28] = float("inf"), float("nan"), float("-inf")
    d["a"][3, 4, 100] = float("nan")
    out = run_project(tts, d, row_stream=of, stream_adapter=sa, odt=odt)
    good = (adapter != 1) & (adapter != 3)
    assert torch.equal(out[good], clean[good]) and out[adapter == 3].isnan().all()
    one, ref = out[adapter == 1], clean[adapter == 1]
    odd = torch.zeros(n, dtype=torch.bool, device="cuda")
    odd[[5, 7, n - 1]] = True
    assert one[:, odd].isfinite().sum() == 0 and one[:, 7].isnan().all() and torch.equal(one[:, ~odd], ref[:, ~odd])
    for r in (0, 17, int((of >= 0).sum()) - 1):
        d = dict(c, x=c["x"].clone())
        if xdt == "bf16":
            d["x"][r, 17] = float("nan")
        else:
            d["x_scale"] = c["x_scale"].clone()
            d["x_scale"][r] = float("nan")
        out = run_project(tts, d, row_stream=of, stream_adapter=sa, odt=odt)
        rest = torch.arange(of.numel(), device="cuda") != r
        assert out[r].isnan().all() and torch.equal(out[rest], clean[rest])


@pytest.mark.parametrize("path", list(PATHS))
@pytest.mark.parametrize("odt", ["f32", "bf16"])
def test_adapters_beside_no_shared_weights(tts, path, odt):  # noqa: F811
    """W = 0: the output is the adapter's part alone, so its 2-norm shows how x A^T was held."""
    c, of, sa, adapter = batch(path, "bf16", 50)
    c["w"].zero_()
    out = run_project(tts, c, row_stream=of, stream_adapter=sa, odt=odt)
    y, _ = R.project(c["x"], c["w"], c["a"], c["b"], c["rank"], c["scale"], adapter.cpu())
    live = of >= 0
    assert (out[live].double() - y[live]).norm() <= (1e-6 if odt == "f32" else 2.0 ** -8) * y[live].norm()


@pytest.mark.parametrize("path", list(PATHS))
@pytest.mark.parametrize("xdt", ["bf16", "e4m3"])
def test_a_poisoned_workspace_of_more_rows(tts, path, xdt):  # noqa: F811
    c, of, sa, adapter = batch(path, xdt, 60)
    rows, k = c["x"].shape
    pool = tts.adapters(c["a"], c["b"], rank=c["rank"], scale=c["scale"])
    ws = tts.project_workspace(rows + 100, c["w"].shape[0], k, xdt, pool)
    first = run_project(tts, c, row_stream=of, stream_adapter=sa)
    for fill in (255, 0, 127):    # NaN, 0, and values past any result
        ws.fill_(fill)
        assert torch.equal(run_project(tts, c, row_stream=of, stream_adapter=sa, ws=ws), first)
    few = rows - rows // 8
    d = dict(c, x=c["x"][:few], x_scale=None if c["x_scale"] is None else c["x_scale"][:few])
    ws.fill_(255)
    check_project(d, run_project(tts, d, row_stream=of[:few].contiguous(), stream_adapter=sa, ws=ws), adapter[:few], dead=of[:few] < 0)


@pytest.mark.parametrize("path", list(PATHS))
@pytest.mark.parametrize("xdt,odt", [("bf16", "bf16"), ("e4m3", "f32")])
def test_requests_replayed_and_on_two_streams(tts, path, xdt, odt):  # noqa: F811
    c, of, sa, adapter = batch(path, xdt, 70)
    rows, k = c["x"].shape
    n = c["w"].shape[0]
    eager = run_project(tts, c, row_stream=of, stream_adapter=sa, odt=odt)
    pool = tts.adapters(c["a"], c["b"], rank=c["rank"], scale=c["scale"])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [tts.project_workspace(rows, n, k, xdt, pool) for _ in streams]
    outs = [torch.zeros_like(eager) for _ in streams]
    maps = [(of.clone(), sa.clone()) for _ in streams]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=streams[0]):
        run_project(tts, c, row_stream=maps[0][0], stream_adapter=maps[0][1], ws=spaces[0], out=outs[0], stream=streams[0])
    for _ in range(4):
        for o in outs:
            o.fill_(-77.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            for _ in range(3):
                graph.replay()
        with torch.cuda.stream(streams[1]):
            for _ in range(5):
                run_project(tts, c, row_stream=maps[1][0], stream_adapter=maps[1][1], ws=spaces[1], out=outs[1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager)
    # another batch in the same graph: other requests, other adapters, more rows of none
    maps[0][0].copy_((of + 1).clamp(max=sa.numel() - 1) * (of >= 0) - (torch.arange(rows, device="cuda") % 9 == 4).to(I32) * 1000)
    maps[0][1].copy_(sa.flip(0))
    outs[0].fill_(-77.0)
    dead = maps[0][0] < 0
    now = torch.where(dead, -1, maps[0][1][maps[0][0].clamp(min=0).long()])
    with torch.cuda.stream(streams[0]):
        graph.replay()
    torch.cuda.synchronize()
    check_project(c, outs[0], now, dead=dead, odt=odt)


@pytest.mark.parametrize("rows,n,k,streams", [(1, 1, 8, 1), (200, 1, 8, 200), (200, 1, 8, 5), (400, 5, 24, 7), (1100, 3400, 8, 9),
                                              (1100, 3400, 40, 9), (257, 9700, 16, 2)])
@pytest.mark.parametrize("xdt,rank_max", [("bf16", 8), ("e4m3", 24), ("bf16", None)])
def test_the_smallest_k_and_n(tts, rows, n, k, streams, xdt, rank_max):  # noqa: F811
    if xdt == "e4m3":
        k = -(-k // 16) * 16
    c = project_case(rows + k, rows, n, k, xdt, None if rank_max is None else 3, rank_max)
    of = (torch.arange(rows, device="cuda") * streams // rows).to(I32)
    sa = ints([i % 4 - 1 for i in range(streams)])
    out = run_project(tts, c, row_stream=of, stream_adapter=None if rank_max is None else sa, pad=1)
    check_project(c, out, None if rank_max is None else sa[of.long()])


@pytest.mark.parametrize("streams", [70000, 60, None])   # on the CUDA cores, on pairs, no adapters
def test_outputs_past_32_bit_offsets(tts, streams):  # noqa: F811
    rows, n, k = 70000, 32768, 64
    g = gen(80)
    x, w = randn(g, rows, k, dt="bf16"), randn(g, n, k, dt="bf16", std=0.05)
    a, b = randn(g, 5, 8, k, dt="bf16", std=0.1), randn(g, 5, n, 8, dt="bf16", std=0.2)
    out = torch.full((rows, n), -77.0, dtype=torch.bfloat16, device="cuda")
    of = sa = pool = ws = None
    if streams is not None:
        of = (torch.arange(rows, device="cuda") * streams // rows).to(I32)
        of[5::997] = -1
        sa = (torch.arange(streams, device="cuda") % 6 - 1).to(I32)
        pool = tts.adapters(a, b)
        ws = tts.project_workspace(rows, n, k, "bf16", pool)
    tts.tts_project_rows(x, w, out, ws, adapters=pool, stream_adapter=sa, row_stream=of)
    at = torch.cat([torch.arange(0, rows, 1777, device="cuda"), torch.arange(rows - 40, rows, device="cuda"),
                    torch.arange(5, rows, 9970, device="cuda")])
    adapter = torch.full((at.numel(),), -1) if of is None else torch.where(of[at] >= 0, sa[of[at].clamp(min=0).long()], -1).cpu()
    y, mass = R.project(x[at], w, a, b, [8] * 5, [1.0] * 5, adapter)
    dead = torch.zeros(at.numel(), dtype=torch.bool, device="cuda") if of is None else of[at] < 0
    assert close(out[at][~dead], y[~dead], mass[~dead], k, 8, "bf16") and (out[at][dead] == -77.0).all()
    assert streams is None or dead.any()
