"""The operators of a step that serves many requests at once, as cases that can be timed.

A pass is what a user's program does with one operator: the residual's addition and the norm
(``norm``), the shared projection with every request's own low-rank adapter (``project``), block
tables and slot maps from request lengths (``plan``: two steps, so that pages come and go), and
rows written into the cache by such a slot map (``slots``).  With ``own`` false, ``run`` computes
them from elementary torch operations in 32 bits (64 where a value sits next to a rounding
border); with ``own`` true it makes the library's calls.  ``exact`` restates each computed one from
its definition in 64 bits.

Shapes are those of the talker (hidden 2048, 16 query and 8 kv heads of 128, an MLP of 6144) and of
its neighbours.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
BYTES = {"f32": 4, "bf16": 2, "e4m3": 1, "i8": 1}
TOP = {"i8": 127.0, "e4m3": 448.0}   # the largest code
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _norm(name, rows, n, x, res, out):
    return {"name": name, "op": "norm", "rows": rows, "n": n, "x": x, "res": res, "out": out}


def _project(name, rows, streams, n, k, x, out, pool, rank, mixed=True, dead=0):
    return {"name": name, "op": "project", "rows": rows, "streams": streams, "n": n, "k": k, "x": x, "out": out,
            "pool": pool, "rank": rank, "mixed": mixed, "dead": dead}


def _plan(name, decode, prompts, longest, page, capacity, t=0):
    return {"name": name, "op": "plan", "decode": decode, "prompts": prompts, "longest": longest, "page": page,
            "capacity": capacity, "t": t}


def _slots(name, rows, src, kv, page, hkv=8, d=128, dead=0):
    return {"name": name, "op": "slots", "rows": rows, "src": src, "kv": kv, "page": page, "hkv": hkv, "d": d,
            "dead": dead}


def listed():
    return [
        # the residual stream of 32 decoding streams after a projection: latency
        _norm("norm 32 rows bf16", 32, 2048, "f32", "f32", "bf16"),
        # a batch of prompts, rows rounded to eight bits for the next projection
        _norm("norm prompts e4m3", 6001, 2048, "bf16", "bf16", "e4m3"),
        # a width that is no power of two, f32 throughout
        _norm("norm odd f32", 1021, 5000, "f32", "f32", "f32"),
        # one request's token through a small projection: latency
        _project("project one token", 1, 1, 2048, 1024, "bf16", "f32", 4, 8),
        # q, k and v of 32 decoding requests with a speaker's adapter each
        _project("project decode bf16", 32, 32, 4096, 2048, "bf16", "f32", 48, 16, mixed=False),
        # gate and up of 96 decoding requests from 8-bit rows and weights, adapters of many ranks
        _project("project decode e4m3", 96, 96, 12288, 2048, "e4m3", "bf16", 64, 64),
        # prompts of seven requests, q, k and v
        _project("project prompts bf16", 4093, 7, 4096, 2048, "bf16", "bf16", 12, 32, mixed=False, dead=3),
        # prompts of many requests through gate and up in eight bits
        _project("project prompts e4m3", 6000, 40, 12288, 2048, "e4m3", "bf16", 24, 16),
        # two decode steps of 64 requests, eight of which come or go: latency
        _plan("plan decode", 56, 4, 40, 16, 4096),
        # two steps of a busy server: prompts beside decoding requests
        _plan("plan prompts", 384, 64, 1200, 16, 4096),
        # one decode step's rows of 64 requests
        _slots("slots decode bf16", 64, "f32", "bf16", 16, dead=2),
        # a packed batch of prompts from a bf16 projection into 8-bit pages
        _slots("slots prompts e4m3", 16001, "bf16", "e4m3", 16, dead=30),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "project", "project", "project", "project", "plan", "slots"])
    if op == "norm":
        rows = _log(rng, 1, 6001)
        c = _norm("", rows, 8 * _log(rng, 8, 1024) if rows < 2000 else 8 * _log(rng, 8, 256), rng.choice(["f32", "bf16"]),
                  rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16", "e4m3"]))
    elif op == "project":
        rows = _log(rng, 1, 6000)
        x = rng.choice(["bf16", "bf16", "e4m3"])
        streams = rows if rng.random() < 0.4 and rows <= 256 else _log(rng, 1, min(rows, 64))
        c = _project("", rows, streams, _log(rng, 16, 12288 if rows < 1000 else 6000),
                     16 * _log(rng, 4, 256 if rows < 1000 else 128), x, rng.choice(["f32", "bf16"]), _log(rng, 1, 48),
                     8 * rng.choice([1, 2, 2, 3, 4, 4, 8, 16]), rng.random() < 0.5, rng.choice([0, 0, rng.randint(0, rows // 2)]))
    elif op == "plan":
        page = rng.choice([1, 8, 16, 64, 256])
        t = rng.choice([0, 0, 0, 8, 64])
        c = _plan("", _log(rng, 1, 384), _log(rng, 1, 64), t or _log(rng, 1, 1200), page, rng.choice([2048, 4096]), t)
    else:
        rows = _log(rng, 1, 12000)
        c = _slots("", rows, rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16", "i8", "e4m3"]),
                   rng.choice([0, 8, 16, 64, 256]), rng.choice([2, 8, 8, 5]), rng.choice([64, 128, 128]),
                   min(rows - 1, rng.choice([0, 1, 7])))
    return {k: v for k, v in c.items() if k != "name"}


def _lengths(c):
    """Rows of each request, which add up to the case's live rows: ragged around the mean."""
    live, n = c["rows"] - c["dead"], c["streams"]
    if n == c["rows"]:
        return [1] * n
    w = [0.25 + (i * 0.6180339887 + 0.3) % 1.0 for i in range(n)]
    total, cut = sum(w), [0]
    for x in w:
        cut.append(cut[-1] + x)
    at = [int(round(x * live / total)) for x in cut]
    return [b - a for a, b in zip(at, at[1:])]


def _ranks(c):
    """Ranks of the pool's adapters: the largest, or with `mixed` all kinds up to it."""
    return [max(1, c["rank"] - (i * 5) % c["rank"]) if c["mixed"] else c["rank"] for i in range(c["pool"])]


def _adapter_of(c):
    """Each request's adapter; every ninth has none."""
    return [-1 if i % 9 == 8 else (i * 7 + 3) % c["pool"] for i in range(c["streams"])]


def _prompt_rows(c):
    """Rows of the two groups of requests that come and go."""
    return [max(1, int(c["longest"] * (0.1 + 0.9 * ((i * 0.7548776662 + 0.2) % 1.0)))) for i in range(2 * c["prompts"])]


def _plan_rows(c):
    return c["decode"] + max(sum(_prompt_rows(c)[: c["prompts"]]), sum(_prompt_rows(c)[c["prompts"]:]))


def work(c):
    if c["op"] == "norm":
        n = c["rows"] * c["n"]
        return {"bytes": n * (BYTES[c["x"]] + 2 * BYTES[c["res"]] + BYTES[c["out"]]) + 4 * c["n"]
                + (4 * c["rows"] if c["out"] == "e4m3" else 0), "flops": n * (7 if c["out"] == "e4m3" else 5)}
    if c["op"] == "project":
        live, n, k = c["rows"] - c["dead"], c["n"], c["k"]
        if c["streams"] == c["rows"]:
            live = c["rows"]
        rank, of, rows = _ranks(c), _adapter_of(c), _lengths(c)
        used = {a for a, m in zip(of, rows) if a >= 0 and m}
        scales = 4 * (live + n) if c["x"] == "e4m3" else 0
        return {"bytes": (live + n) * k * BYTES[c["x"]] + scales + live * n * BYTES[c["out"]]
                + sum(rank[a] for a in used) * (n + k) * 2 + 8 * live,
                "flops": 2 * live * n * k + sum(2 * m * rank[a] * (n + k) for a, m in zip(of, rows) if a >= 0)}
    if c["op"] == "plan":
        b = c["decode"] + 2 * c["prompts"]
        pages = sum(-(-m // c["page"]) for m in _prompt_rows(c))
        # a step reads two words a stream and writes one, and a map entry of 16 bytes a row; a page
        # that comes or goes is read and written once each
        return {"bytes": 2 * (12 * b + 16 * _plan_rows(c)) + 16 * pages, "flops": 0}
    rows, e = c["rows"] - c["dead"], c["hkv"] * c["d"] * 2
    return {"bytes": rows * (e * (BYTES[c["src"]] + BYTES[c["kv"]]) + 8 + (8 * c["hkv"] if c["kv"] in TOP else 0)),
            "flops": rows * e * (4 if c["kv"] in TOP else 0)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _quantised(x):
    """Rows in e4m3 and their scales."""
    s = (x.abs().amax(-1) / TOP["e4m3"]).clamp_min(1e-12)
    return (x / s[:, None]).clamp(-448, 448).to(DT["e4m3"]), s


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(c, seed):
    g, s = _gen(seed), {"case": c}
    if c["op"] == "norm":
        # a few channels of a residual stream are far larger than the others
        big = torch.exp(1.5 * _randn(g, c["n"]).clamp(-3, 3))
        s["x"] = _randn(g, c["rows"], c["n"], dtype=DT[c["x"]])
        s["res"] = (_randn(g, c["rows"], c["n"]) * big).to(DT[c["res"]])
        s["gamma"] = torch.rand(c["n"], generator=g, device=DEV) + 0.5
        s["sum"] = torch.empty_like(s["res"])
        s["out"] = torch.zeros(c["rows"], c["n"], dtype=DT[c["out"]], device=DEV)
        s["scale"] = torch.zeros(c["rows"], device=DEV) if c["out"] == "e4m3" else None
        return s
    if c["op"] == "project":
        n, k, r = c["n"], c["k"], c["rank"]
        x, w = _randn(g, c["rows"], k), _randn(g, n, k, std=0.02)
        if c["x"] == "e4m3":
            (s["x"], s["xs"]), (s["w"], s["ws"]) = _quantised(x), _quantised(w)
        else:
            s["x"], s["w"] = x.to(DT[c["x"]]), w.to(DT[c["x"]])
        # an adapter of a smaller rank leaves the rest of its place in the pool unused
        s["a"] = _randn(g, c["pool"], r, k, dtype=torch.bfloat16, std=k ** -0.5)
        s["b"] = _randn(g, c["pool"], n, r, dtype=torch.bfloat16, std=0.05)
        s["rank"], s["alpha"] = _ints(_ranks(c)), 1.0 + torch.rand(c["pool"], generator=g, device=DEV)
        s["adapter"] = _ints(_adapter_of(c))
        s["row_stream"] = None
        if c["streams"] != c["rows"]:
            of = torch.repeat_interleave(torch.arange(c["streams"]), torch.tensor(_lengths(c)))
            of = torch.cat([of, torch.full((c["rows"] - of.numel(),), -1)])
            s["row_stream"] = of.to(DEV, torch.int32)
        s["out"] = torch.zeros(c["rows"], n, dtype=DT[c["out"]], device=DEV)
        return s
    if c["op"] == "plan":
        return _prepare_plan(c, g, s)
    page = c["page"] or 256
    need = -(-c["rows"] // page) + 3
    for key in ("k", "v"):
        s[key] = torch.zeros(need, c["hkv"], page, c["d"], dtype=DT[c["kv"]], device=DEV)
        s[key + "_scale"] = torch.zeros(need, c["hkv"], page, device=DEV) if c["kv"] in TOP else None
    s["pages"] = need
    s["src"] = (_randn(g, c["rows"], 2 * c["hkv"] * c["d"]) * torch.exp(_randn(g, c["rows"], 1))).to(DT[c["src"]])
    # rows fill their pages in order, the pages lie anywhere
    r = torch.arange(c["rows"], device=DEV)
    slot = torch.randperm(need, generator=g, device=DEV)[r // page] * page + r % page
    s["slot"] = torch.where(r < c["rows"] - c["dead"], slot, -1)
    return s


def _prepare_plan(c, g, s):
    page, cap = c["page"], c["capacity"]
    b, per = c["decode"] + 2 * c["prompts"], cap // page
    past = torch.zeros(b, dtype=torch.int64, device=DEV)
    past[: c["decode"]] = torch.randint(0, cap // 2, (c["decode"],), generator=g, device=DEV)
    rows = _prompt_rows(c)
    new = torch.ones(2, b, dtype=torch.int32, device=DEV)
    x, y = slice(c["decode"], c["decode"] + c["prompts"]), slice(c["decode"] + c["prompts"], b)
    # the first step's prompts end in the second, whose prompts end in the next pass
    new[0, x], new[0, y] = _ints(rows[: c["prompts"]]), -1
    new[1, y], new[1, x] = _ints(rows[c["prompts"]:]), -1
    held = (past + page - 1) // page
    pages = b * per // 2 + 3 * b + sum(-(-m // page) for m in rows)
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    first = torch.cumsum(held, 0) - held
    i = torch.arange(per, device=DEV)
    s["table"] = torch.where(i < held[:, None], perm[(first[:, None] + i).clamp(max=pages - 1)], -1).to(torch.int32)
    s["free"] = torch.cat([perm[held.sum():], perm[: held.sum()]]).contiguous()
    s["n_free"] = (pages - held.sum()).to(torch.int32).reshape(1)
    s["past"], s["new"], s["pages"] = past.to(torch.int32), new, pages
    n = b * c["t"] if c["t"] else _plan_rows(c) + 5
    s["max_rows"] = n
    s["maps"] = [{"n_rows": torch.zeros(b, dtype=torch.int32, device=DEV),
                  "row_start": torch.zeros(b + 1, dtype=torch.int32, device=DEV),
                  "row_stream": torch.zeros(n, dtype=torch.int32, device=DEV),
                  "row_pos": torch.zeros(n, dtype=torch.int32, device=DEV),
                  "row_slot": torch.zeros(n, dtype=torch.int64, device=DEV)} for _ in range(2)]
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    return {"norm": _plain_norm, "project": _plain_project, "plan": _plain_plan, "slots": _plain_slots}[s["case"]["op"]](s)


def _e4m3_code(x):
    """The nearest code to each exact quotient (given in 64 bits), ties to the even one."""
    m, e = torch.frexp(x)
    e = torch.clamp(e, min=-5)
    step = torch.exp2((e - 4).double()).float().double()      # (a power of two: exact in f32)
    return ((x / step).round() * step).clamp(-448, 448)


def _plain_norm(s):
    c = s["case"]
    h = (s["res"].float() + s["x"].float()).to(DT[c["res"]])
    s["sum"].copy_(h)
    h = h.float()
    y = h * (1.0 / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS)) * s["gamma"]
    if c["out"] != "e4m3":
        return {"sum": s["sum"], "out": y.to(DT[c["out"]])}
    scale = y.abs().amax(-1) * (1.0 / 448.0)
    q = y.double() / scale[:, None].double()
    return {"sum": s["sum"], "out": _e4m3_code(q).to(DT["e4m3"]), "scale": scale}


def _plain_project(s):
    c = s["case"]
    x = s["x"].float()
    y = x @ s["w"].float().T
    if c["x"] == "e4m3":
        x = x * s["xs"][:, None]
        y = y * s["xs"][:, None] * s["ws"]
    of = torch.arange(c["rows"], device=DEV) if s["row_stream"] is None else s["row_stream"].long()
    a = torch.where(of >= 0, s["adapter"][of.clamp(min=0)].long(), -1)
    # every adapter's low-rank rows side by side; a row keeps those of its own
    v = (x @ s["a"].float().flatten(0, 1).T).unflatten(1, (c["pool"], c["rank"]))
    keep = (a[:, None] == torch.arange(c["pool"], device=DEV))[..., None] & \
        (torch.arange(c["rank"], device=DEV) < s["rank"][:, None])
    v = torch.where(keep, v * s["alpha"][:, None], 0.0)
    y = y + v.flatten(1) @ s["b"].float().transpose(1, 2).flatten(0, 1)
    s["out"].copy_(torch.where((of >= 0)[:, None], y.to(DT[c["out"]]), s["out"]))
    return s["out"]


def _plain_step(s, step):
    c, m = s["case"], s["maps"][step]
    page, table = c["page"], s["table"].long()
    b, per = table.shape
    free, n_free, new, past = s["free"].long(), s["n_free"].long(), s["new"][step].long(), s["past"].long()
    held = (table >= 0) & (table < s["pages"])
    # pages of requests that ended go on the free list, in order
    give = held & (new < 0)[:, None]
    at = n_free + torch.cumsum(give.flatten(), 0) - 1
    more = torch.cat([free, free[:1]])
    more.scatter_(0, torch.where(give.flatten(), at, s["pages"]), table.flatten())
    free, n_free = more[:-1], n_free + give.sum()
    table = torch.where(give, -1, table)
    # requests in order take pages from the list's end, as long as they last
    i = torch.arange(per, device=DEV)
    valid = (new > 0) & (past + new <= c["capacity"])
    want = valid[:, None] & ~held & (i >= (past // page)[:, None]) & (i <= ((past + new - 1) // page)[:, None])
    need = want.sum(1)
    upto = torch.cumsum(need, 0)
    ok = valid & ((need == 0) | (upto <= n_free))
    if c["t"]:
        ok = ok & (new <= c["t"])
    else:
        ok = ok & (torch.cumsum(torch.where(ok, new, 0), 0) <= s["max_rows"])
    k = (upto - need)[:, None] + torch.cumsum(want, 1) - 1
    got = want & ok[:, None]
    table = torch.where(got, free[(n_free - 1 - k).clamp(min=0)], table)
    n = torch.where(ok, new, 0)
    s["free"].copy_(free)
    s["n_free"].copy_(n_free - torch.where(ok, need, 0).sum())
    s["table"].copy_(table)
    r = torch.arange(s["max_rows"], device=DEV)
    if c["t"]:
        start = torch.arange(b + 1, device=DEV) * c["t"]
        of = r // c["t"]
        live = r % c["t"] < n[of]
    else:
        start = torch.cat([torch.zeros_like(n[:1]), torch.cumsum(n, 0)])
        of = torch.searchsorted(start[1:].contiguous(), r, right=True)
        live = r < start[-1]
    of = of.clamp(max=b - 1)
    pos = past[of] + r - start[of]
    slot = table[of, (pos // page).clamp(0, per - 1)] * page + pos % page
    m["n_rows"].copy_(n)
    m["row_start"].copy_(start)
    m["row_stream"].copy_(torch.where(live, of, -1))
    m["row_pos"].copy_(torch.where(live, pos, 0))
    m["row_slot"].copy_(torch.where(live, slot, -1))
    return m


def _plan_state(s):
    return {"table": s["table"], "free": s["free"], "n_free": s["n_free"]}


def _plain_plan(s):
    return {"first": _plain_step(s, 0), "second": _plain_step(s, 1), "state": _plan_state(s)}


def _plain_slots(s):
    c = s["case"]
    page = c["page"] or 256
    src = s["src"].float().reshape(c["rows"], 2, c["hkv"], c["d"])
    # rows without a slot go to a page behind the pool
    slot = torch.where(s["slot"] >= 0, s["slot"], s["pages"] * page)
    at, off, g = (slot // page)[:, None], (slot % page)[:, None], torch.arange(c["hkv"], device=DEV)
    got = {}
    for i, key in enumerate(("k", "v")):
        x = src[:, i]
        if c["kv"] in TOP:
            sc = x.abs().amax(-1) * (1.0 / TOP[c["kv"]])
            x = x.double() / sc[..., None].double()
            x = x.round().clamp(-127, 127) if c["kv"] == "i8" else _e4m3_code(x)
            got[key + "_scale"] = _put(s[key + "_scale"], (at, g, off), sc)
        got[key] = _put(s[key], (at, g, off), x.to(DT[c["kv"]]))
    return got


def _put(cache, at, x):
    """Rows x at `at` of the cache, whose last page here is for rows that have no slot."""
    raw, y = (cache.view(torch.uint8), x.view(torch.uint8)) if x.dtype == torch.float8_e4m3fn else (cache, x)
    wide = torch.cat([raw, raw[:1]])
    wide[at] = y
    raw.copy_(wide[:-1])
    return cache


def _own(s):
    from autoregressive_codebook_tts_gb300 import tts
    c = s["case"]
    if c["op"] == "norm":
        tts.tts_add_rms_norm(s["x"], s["res"], s["sum"], s["gamma"], EPS, s["out"], out_scale=s["scale"])
        got = {"sum": s["sum"], "out": s["out"]}
        return dict(got, scale=s["scale"]) if c["out"] == "e4m3" else got
    if c["op"] == "project":
        if "pool" not in s:
            s["pool"] = tts.adapters(s["a"], s["b"], rank=s["rank"], scale=s["alpha"])
            s["work"] = tts.project_workspace(c["rows"], c["n"], c["k"], c["x"], s["pool"])
        tts.tts_project_rows(s["x"], s["w"], s["out"], s["work"], x_scale=s.get("xs"), w_scale=s.get("ws"),
                             adapters=s["pool"], stream_adapter=s["adapter"], row_stream=s["row_stream"])
        return s["out"]
    if c["op"] == "plan":
        if "desc" not in s:
            s["desc"] = tts.kv_desc(s["table"].shape[0], 16, 8, 128, c["capacity"], "bf16", paged=True,
                                    page_size=c["page"], n_pages=s["pages"], block_table=s["table"])
        for step, m in enumerate(s["maps"]):
            tts.tts_page_plan(s["desc"], s["table"], s["free"], s["n_free"], s["past"], s["new"][step], m["n_rows"],
                              m["row_start"], m["row_stream"], m["row_pos"], m["row_slot"], T=c["t"])
        return {"first": s["maps"][0], "second": s["maps"][1], "state": _plan_state(s)}
    if "desc" not in s:
        page = c["page"] or 256
        s["table"] = torch.zeros(1, 1, dtype=torch.int32, device=DEV) if c["page"] else None
        s["desc"] = tts.kv_desc(s["pages"] if not c["page"] else 1, c["hkv"], c["hkv"], c["d"], page, c["kv"],
                                window_quantum=page, paged=c["page"] > 0, page_size=c["page"], n_pages=s["pages"],
                                block_table=s["table"])
        s["cache"] = tts.kv_cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    kd = c["hkv"] * c["d"]
    tts.tts_kv_write_slots(s["src"][:, :kd], s["src"][:, kd:], s["cache"], s["desc"], s["slot"])
    return {k: s[k] for k in ("k", "v", "k_scale", "v_scale") if s[k] is not None}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(c, seed):
    if c["op"] == "plan":
        return None   # whole numbers
    s = prepare(c, seed)
    return {"norm": _exact_norm, "project": _exact_project, "slots": _exact_slots}[c["op"]](c, s)


_E4M3 = sorted({(m / 8 + (e > 0)) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8) if (e, m) != (15, 7)})


def _nearest(x):
    """The nearest code by search among all of them; a tie goes to the even one."""
    grid = torch.tensor(_E4M3, device=DEV, dtype=torch.float64)
    mid = (grid[1:] + grid[:-1]) / 2
    low, high = torch.searchsorted(mid, x.abs()), torch.searchsorted(mid, x.abs(), right=True)
    i = torch.where((low != high) & (low % 2 == 1), high, low)
    return torch.sign(x) * grid[i]


def _exact_norm(c, s):
    h = (s["res"].double() + s["x"].double()).float().to(DT[c["res"]]).double()
    y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / c["n"] + EPS) * s["gamma"].double()
    if c["out"] != "e4m3":
        return {"sum": h, "out": y}
    scale = y.abs().amax(-1) / 448.0
    return {"sum": h, "out": _nearest(y / scale[:, None]), "scale": scale}


def _exact_project(c, s):
    x, w = s["x"].float().double(), s["w"].float().double()
    if c["x"] == "e4m3":
        x, w = x * s["xs"].double()[:, None], w * s["ws"].double()[:, None]
    out = s["out"].double()
    rank, r = _ranks(c), 0
    for a, m in zip(_adapter_of(c), _lengths(c)):
        xs = x[r: r + m]
        y = xs @ w.T
        if a >= 0:
            v = xs @ s["a"][a, : rank[a]].double().T
            y = y + float(s["alpha"][a]) * (v @ s["b"][a, :, : rank[a]].double().T)
        out[r: r + m] = y
        r += m
    return out


def _exact_slots(c, s):
    page, got = c["page"] or 256, {}
    x = s["src"].double().view(c["rows"], 2, c["hkv"], c["d"])[: c["rows"] - c["dead"]]
    slot = s["slot"][: c["rows"] - c["dead"]]
    for i, key in enumerate(("k", "v")):
        y = x[:, i]
        if c["kv"] in TOP:
            scale = torch.zeros(s["pages"] * page, c["hkv"], dtype=torch.float64, device=DEV)
            sc = y.abs().amax(-1).float() * torch.tensor(1.0 / TOP[c["kv"]], device=DEV)
            scale[slot] = sc.double()
            got[key + "_scale"] = scale.view(s["pages"], page, c["hkv"]).transpose(1, 2)
            y = y / sc.double()[..., None]
            y = y.round().clamp(-127, 127) if c["kv"] == "i8" else _nearest(y)
        elif c["kv"] == "bf16":
            y = y.float().to(torch.bfloat16).double()
        cache = torch.zeros(s["pages"] * page, c["hkv"], c["d"], dtype=torch.float64, device=DEV)
        cache[slot] = y
        got[key] = cache.view(s["pages"], page, c["hkv"], c["d"]).transpose(1, 2)
        if c["kv"] == "i8":
            got[key] = got[key].to(torch.int8)
    return got
