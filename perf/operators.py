"""The operators of drafted decoding over a quantised cache, as cases that can be timed.

A pass is one call of a user's program: rotary positions of projection rows (``rope``,
``table``), rows written into a quantised cache and read back (``kv``), attention of a tree
of drafted tokens over a cache (``tree``), and the accepted path moved to the front of the
tree's rows (``commit``).  With ``own`` false, ``run`` computes them from elementary torch
operations in 32 bits (64 where a value sits next to a rounding border); with ``own`` true
it makes the library's calls.  ``exact`` restates each from its definition in 64 bits.

Shapes are those of the talker (16 query heads, 8 kv heads of 128, 4096 positions) and of
its neighbours: 64-wide heads, other groupings, pages of the paged workload.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
CACHE_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"i8": 127.0, "e4m3": 448.0}   # the largest code
BYTES = {"f32": 4, "bf16": 2, "i8": 1, "e4m3": 1}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _rope(name, rows, dtype, out_dtype, hq=16, hkv=8, d=128, rot=128, inter=False, norm=True, max_pos=4096):
    return {"name": name, "op": "rope", "rows": rows, "dtype": dtype, "out_dtype": out_dtype, "hq": hq, "hkv": hkv,
            "d": d, "rot": rot, "inter": inter, "norm": norm, "max_pos": max_pos}


def _table(name, max_pos, rot, kind, factor, original, attn_scale, base=1e6):
    return {"name": name, "op": "table", "max_pos": max_pos, "rot": rot, "kind": kind, "factor": factor,
            "original": original, "attn_scale": attn_scale, "base": base}


def _kv(name, b, t, kv, src, out, lo, hi, hkv=8, d=128, page=0, window=False, ragged=False):
    return {"name": name, "op": "kv", "b": b, "t": t, "kv": kv, "src": src, "out": out, "lo": lo, "hi": hi,
            "hkv": hkv, "d": d, "page": page, "window": window, "ragged": ragged}


def _tree(name, b, t, kv, q, lo, hi, hq=16, hkv=8, d=128, page=0, chain=False, ragged=False):
    return {"name": name, "op": "tree", "b": b, "t": t, "kv": kv, "q": q, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv,
            "d": d, "page": page, "chain": chain, "ragged": ragged}


def _commit(name, b, t, kv, capacity, hkv=8, d=128, page=0):
    return {"name": name, "op": "commit", "b": b, "t": t, "kv": kv, "capacity": capacity, "hkv": hkv, "d": d,
            "page": page}


def listed():
    return [
        # one decode step's q and k rows of 32 streams: latency
        _rope("rope 32 rows f32", 32, "f32", "f32"),
        # a prompt's rows, a quarter-rotated interleaved layout, bf16 out for the attention
        _rope("rope prompt bf16", 8191, "f32", "bf16", rot=32, inter=True, max_pos=16384),
        # a table for a window eight times the original, built when a model is loaded
        _table("table by parts", 32768, 128, "parts", 8.0, 4096, 1.2079),
        # one decode step's new rows of 32 streams into an int8 cache, read back
        _kv("kv step i8", 32, 1, "i8", "f32", "f32", 64, 2047),
        # a ragged prompt chunk into paged e4m3 rows, then the window for a bf16 prefill
        _kv("kv chunk e4m3 paged", 4, 509, "e4m3", "f32", "bf16", 256, 3000, page=16, window=True, ragged=True),
        # a large chunk from a bf16 projection
        _kv("kv chunk i8", 16, 1024, "i8", "bf16", "bf16", 0, 2500, window=True),
        # a short chain of drafts of one stream, f32 throughout: latency
        _tree("tree chain f32", 1, 5, "f32", "f32", 255, 255, chain=True),
        # the single-token form of 32 ragged streams over an int8 cache
        _tree("tree token i8", 32, 1, "i8", "bf16", 64, 2048, chain=True),
        # sixteen drafted nodes of 8 streams over 16-row pages of bf16
        _tree("tree paged bf16", 8, 16, "bf16", "bf16", 3264, 3907, page=16),
        # the widest trees of 32 streams over an e4m3 cache
        _tree("tree wide e4m3", 32, 63, "e4m3", "bf16", 1500, 4000, ragged=True),
        # one stream's accepted path
        _commit("commit one f32", 1, 7, "f32", 256),
        # 32 streams' accepted paths, 16-row pages
        _commit("commit batch bf16", 32, 64, "bf16", 512, page=16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    hq, hkv = rng.choice([(16, 8), (16, 8), (8, 8), (16, 4), (4, 2), (12, 6)])
    d = rng.choice([128, 128, 64])
    op = rng.choice(["rope", "table", "kv", "kv", "tree", "tree", "tree", "tree", "commit"])
    if op == "rope":
        return _without_name(_rope("", _log(rng, 1, 8191), rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"]),
                                   hq, hkv, d, rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]),
                                   rng.random() < 0.5, rng.random() < 0.6, _log(rng, 64, 32768)))
    if op == "table":
        return _without_name(_table("", _log(rng, 16, 32768), 2 * rng.randint(2, 64),
                                    rng.choice(["none", "linear", "base", "parts"]), rng.choice([1.0, 2.0, 4.0, 8.0, 11.5]),
                                    rng.choice([1024, 2048, 4096]), round(rng.uniform(0.8, 1.3), 4),
                                    rng.choice([1e4, 5e5, 1e6])))
    page = rng.choice([0, 0, 8, 16, 64, 256])
    if op == "kv":
        t = _log(rng, 1, 1024)
        b = _log(rng, 1, max(1, min(32, 16384 // t)))
        hi = _log(rng, 1, 2500)
        return _without_name(_kv("", b, t, rng.choice(["i8", "e4m3", "i8", "e4m3", "bf16"]), rng.choice(["f32", "bf16"]),
                                 rng.choice(["f32", "bf16"]) if b * (t + hi) < 20000 else "bf16", rng.randint(0, hi), hi, hkv, d, page,
                                 rng.random() < 0.5 and b * (t + hi) < 50000, rng.random() < 0.5))
    if op == "tree":
        t = _log(rng, 1, 64)
        b = _log(rng, 1, 32)
        hi = _log(rng, 1, 4000)
        q = rng.choice(["f32", "bf16", "bf16"])
        kv = rng.choice(["f32", "bf16", "i8", "e4m3"])
        return _without_name(_tree("", b, t, kv, q, rng.randint(0, hi), hi, hq, hkv, d, page, rng.random() < 0.3,
                                   rng.random() < 0.5))
    return _without_name(_commit("", _log(rng, 1, 32), rng.randint(1, 64), rng.choice(["f32", "bf16", "i8"]),
                                 rng.choice([256, 512]), hkv, d, page))


def _without_name(c):
    return {k: v for k, v in c.items() if k != "name"}


def _lens(c):
    """Each stream's committed rows, spread over [lo, hi]."""
    span = c["hi"] - c["lo"]
    return [c["lo"] + int((b * 0.6180339887 + 0.5) % 1.0 * (span + 1)) for b in range(c["b"])]


def _counts(c):
    """Each stream's rows of this pass: all T, or in a ragged batch from T / 2 up."""
    if not c["ragged"]:
        return [c["t"]] * c["b"]
    return [c["t"] - int((b * 0.7548776662) % 1.0 * (c["t"] // 2 + 1)) for b in range(c["b"])]


def _capacity(c):
    need = c["capacity"] if c["op"] == "commit" else c["hi"] + c["t"]
    return (need + 255) // 256 * 256


def work(c):
    if c["op"] == "rope":
        n = c["rows"] * (c["hq"] + c["hkv"]) * c["d"]
        return {"bytes": n * (BYTES[c["dtype"]] + BYTES[c["out_dtype"]]) + c["rows"] * 4
                + min(c["rows"], c["max_pos"]) * c["rot"] * 4 + (8 * c["d"] if c["norm"] else 0),
                "flops": n * (3 + (4 if c["norm"] else 0))}
    if c["op"] == "table":
        return {"bytes": c["max_pos"] * c["rot"] * 4, "flops": c["max_pos"] * c["rot"] * 2}
    if c["op"] == "commit":
        rows = sum(max(1, c["t"] // 4 + b % 3) for b in range(c["b"])) * 2 * c["hkv"]
        per = c["d"] * BYTES[c["kv"]] + (4 if c["kv"] == "i8" else 0)
        return {"bytes": 2 * rows * per, "flops": 0}
    scale = 4 if c["kv"] in TOP else 0
    per = c["hkv"] * 2
    if c["op"] == "kv":
        lens, counts = _lens(c), _counts(c)
        wrote = sum(counts)
        read = sum(n + k for n, k in zip(lens, counts)) if c["window"] else wrote
        row = c["d"] * BYTES[c["kv"]] + scale
        return {"bytes": per * (wrote * (c["d"] * BYTES[c["src"]] + row) + read * (row + c["d"] * BYTES[c["out"]])),
                "flops": per * c["d"] * (4 * wrote + read)}
    lens, counts = _lens(c), _counts(c)
    rows = sum(n + k for n, k in zip(lens, counts))
    seen = sum(k * (n + (k + 1) // 2) for n, k in zip(lens, counts))
    return {"bytes": rows * per * (c["d"] * BYTES[c["kv"]] + scale) + 2 * sum(counts) * c["hq"] * c["d"] * BYTES[c["q"]]
            + sum(counts) * 8 + 8 * c["b"], "flops": 4 * seen * c["hq"] * c["d"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _cache(c, g, pages):
    """K, V and their scales with random rows everywhere: [streams or pages][Hkv][rows][D]."""
    rows = c["page"] or _capacity(c)
    n = pages if c["page"] else c["b"]
    out = {}
    for key in ("k", "v"):
        x = _randn(g, n, c["hkv"], rows, c["d"])
        if c["kv"] in TOP:
            s = (x.abs().amax(-1) / TOP[c["kv"]]).clamp_min(1e-6)
            x = (x / s[..., None]).clamp(-TOP[c["kv"]], TOP[c["kv"]])
            x = (x.round() if c["kv"] == "i8" else x).to(CACHE_DT[c["kv"]])
            out[key + "_scale"] = s
        out[key] = x.to(CACHE_DT[c["kv"]])
    return out


def _pages(c, g, s):
    """A shuffled pool with an eighth more pages than the streams need, and their tables."""
    if not c["page"]:
        return 0
    per = _capacity(c) // c["page"]
    n = c["b"] * per + (c["b"] * per + 7) // 8
    perm = torch.randperm(n, generator=g, device=DEV)
    s["table"] = perm[: c["b"] * per].reshape(c["b"], per).to(torch.int32).contiguous()
    return n


def _trees(c, seed):
    """Each node's ancestors and itself as 64 bits: random trees, parents before children."""
    rng = np.random.RandomState(int(seed) % (1 << 32))
    m = np.zeros((c["b"], c["t"]), np.uint64)
    for b in range(c["b"]):
        for t in range(c["t"]):
            up = m[b, rng.randint(max(0, t - 8), t)] if t and rng.rand() < 0.9 else np.uint64(0)
            m[b, t] = up | (np.uint64(1) << np.uint64(t))
    return torch.from_numpy(m.view(np.int64)).to(DEV)


def prepare(c, seed):
    g = _gen(seed)
    s = {"case": c}
    if c["op"] == "rope":
        width = (c["hq"] + 2 * c["hkv"]) * c["d"]
        s["rows"] = _randn(g, c["rows"], width, dtype=DT[c["dtype"]])
        s["pos"] = torch.randint(0, c["max_pos"], (c["rows"],), generator=g, device=DEV, dtype=torch.int32)
        i = torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64)
        a = torch.arange(c["max_pos"], device=DEV, dtype=torch.float64)[:, None] * torch.pow(1e6, -2.0 * i / c["rot"])
        s["cs"] = torch.stack([a.cos(), a.sin()], -1).float().contiguous()
        for k in ("gq", "gk"):
            s[k] = torch.rand(c["d"], generator=g, device=DEV) + 0.5
        return s
    if c["op"] == "table":
        # a model's own base: another seed is another model
        s["base"] = c["base"] * (1.0 + (int(seed) % 997) / 2000.0)
        return s
    pages = _pages(c, g, s)
    s.update(_cache(c, g, pages))
    s["pages"] = pages
    if c["op"] == "commit":
        cap = _capacity(c)
        s["n_past"] = torch.randint(0, cap - c["t"] + 1, (c["b"],), generator=g, device=DEV, dtype=torch.int32)
        n = [max(1, c["t"] // 4 + b % 3) for b in range(c["b"])]
        n = [min(x, c["t"]) for x in n]
        keys = torch.rand(c["b"], c["t"], generator=g, device=DEV).argsort(1)
        keep = torch.tensor(n, device=DEV)[:, None] > torch.arange(c["t"], device=DEV)
        keys = torch.where(keep, keys, c["t"])
        s["path"] = keys.sort(1).values.to(torch.int32).contiguous()
        s["n_accept"] = torch.tensor(n, dtype=torch.int32, device=DEV)
        return s
    s["n_past"] = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)
    s["count"] = torch.tensor(_counts(c), dtype=torch.int32, device=DEV)
    if c["op"] == "kv":
        # projection rows [k | v], of which a few are far larger than the others
        x = _randn(g, c["b"] * c["t"], 2 * c["hkv"] * c["d"])
        x = x * torch.exp(_randn(g, c["b"] * c["t"], 1))
        s["src"] = x.to(DT[c["src"]])
        n = max(x + y for x, y in zip(_lens(c), _counts(c))) if c["window"] else c["t"]
        for k in ("k_out", "v_out"):
            s[k] = torch.zeros(c["b"], n, c["hkv"], c["d"], dtype=DT[c["out"]], device=DEV)
        return s
    s["q"] = _randn(g, c["b"], c["t"], c["hq"], c["d"], dtype=DT[c["q"]])
    s["mask"] = None if c["chain"] else _trees(c, seed)
    s["out"] = torch.zeros(c["b"], c["t"], c["hq"], c["d"], dtype=DT[c["q"]], device=DEV)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "table": _plain_table, "kv": _plain_kv, "tree": _plain_tree,
            "commit": _plain_commit}[s["case"]["op"]](s)


def _heads(x, h, d):
    return x.reshape(x.shape[0], h, d)


def _plain_rope(s):
    c = s["case"]
    qd, kd = c["hq"] * c["d"], c["hkv"] * c["d"]
    x = s["rows"][:, : qd + kd].float()
    x = _heads(x, c["hq"] + c["hkv"], c["d"])
    if c["norm"]:
        gam = torch.cat([s["gq"].expand(c["hq"], -1), s["gk"].expand(c["hkv"], -1)])
        x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * gam
    cs = s["cs"][s["pos"].long()][:, None]
    co, si = cs[..., 0], cs[..., 1]
    rot, rest = x[..., : c["rot"]], x[..., c["rot"]:]
    if c["inter"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * co - b * si, a * si + b * co], -1).flatten(-2)
    else:
        a, b = rot[..., : c["rot"] // 2], rot[..., c["rot"] // 2:]
        rot = torch.cat([a * co - b * si, a * si + b * co], -1)
    y = torch.cat([rot, rest], -1).to(DT[c["out_dtype"]])
    return {"q": y[:, : c["hq"]].flatten(1), "k": y[:, c["hq"]:].flatten(1)}


def _plain_table(s):
    c = s["case"]
    i = torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64)
    base = torch.full((), s["base"], device=DEV, dtype=torch.float64)
    if c["kind"] == "base":
        base = base * c["factor"] ** (c["rot"] / (c["rot"] - 2.0))
    f = torch.exp(-2.0 * i / c["rot"] * base.log())
    if c["kind"] == "linear":
        f = f / c["factor"]
    if c["kind"] == "parts":
        w = ((c["original"] * f / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        f = f * (w + (1 - w) / c["factor"])
    a = torch.arange(c["max_pos"], device=DEV, dtype=torch.float64)[:, None] * f
    return (torch.stack([a.cos(), a.sin()], -1) * c["attn_scale"]).float()


def _slots(s, pos):
    """The cache rows (of the flattened [n][Hkv][rows]) of positions pos [B][N], [B][N][Hkv]."""
    c = s["case"]
    g = torch.arange(c["hkv"], device=DEV)
    if c["page"]:
        page = torch.gather(s["table"].long(), 1, pos // c["page"])
        return (page[..., None] * c["hkv"] + g) * c["page"] + (pos % c["page"])[..., None]
    b = torch.arange(c["b"], device=DEV)[:, None, None]
    return (b * c["hkv"] + g) * _capacity(c) + pos[..., None]


def _flat(s, key):
    t = s[key]
    return t.reshape(-1, t.shape[-1])


def _values(s, key, slots):
    """The f32 values of the cache rows `slots`."""
    x = _flat(s, key)
    x = (x.view(torch.uint8)[slots].view(x.dtype) if x.dtype == torch.float8_e4m3fn else x[slots]).float()
    return x * s[key + "_scale"].reshape(-1)[slots][..., None] if key + "_scale" in s else x


def _code(x, kv):
    """The nearest code of each exact quotient (given in 64 bits), ties to the even one."""
    if kv == "i8":
        return x.round().clamp(-127, 127)
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), torch.clamp(e - 4, min=-9))
    return ((x / step).round() * step).clamp(-448, 448)


def _plain_kv(s):
    c = s["case"]
    t = torch.arange(c["t"], device=DEV)
    live = t < s["count"][:, None]
    pos = torch.where(live, s["n_past"][:, None].long() + t, 0)
    slots = _slots(s, pos)
    at = slots[live]
    src = s["src"].float().reshape(c["b"], c["t"], 2, c["hkv"], c["d"])
    for i, key in enumerate(("k", "v")):
        x = src[:, :, i][live]
        if c["kv"] in TOP:
            sc = x.abs().amax(-1) / TOP[c["kv"]]
            x = _code(x.double() / sc[..., None].double(), c["kv"])
            s[key + "_scale"].view(-1)[at] = sc
        x = x.to(CACHE_DT[c["kv"]])
        if c["kv"] == "e4m3":
            _flat(s, key).view(torch.uint8)[at] = x.view(torch.uint8)
        else:
            _flat(s, key)[at] = x
    if c["window"]:
        t = torch.arange(s["k_out"].shape[1], device=DEV)
        live = t < (s["n_past"] + s["count"])[:, None]
        slots = _slots(s, torch.where(live, t, 0))
    for key in ("k", "v"):
        s[key + "_out"][live] = _values(s, key, slots[live]).to(DT[c["out"]])
    got = {"k": s["k_out"], "v": s["v_out"]}
    return dict(got, ks=s["k_scale"], vs=s["v_scale"]) if c["kv"] in TOP else got


def _visible(s, n):
    """Which of the first n positions node t of stream b sees, [B][T][n]."""
    c = s["case"]
    j = torch.arange(n, device=DEV)
    u = j - s["n_past"][:, None].long()                                   # [B][n]
    t = torch.arange(c["t"], device=DEV)
    node = (u >= 0) & (u < s["count"][:, None])
    if s["mask"] is None:
        see = u[:, None] <= t[:, None]
    else:
        see = (s["mask"][:, :, None] >> u.clamp(0, 63)[:, None]) & 1 == 1
    return (u < 0)[:, None] | (node[:, None] & see)


def _plain_tree(s):
    c = s["case"]
    n = max(x + y for x, y in zip(_lens(c), _counts(c)))
    slots = _slots(s, torch.arange(n, device=DEV).expand(c["b"], n)).transpose(1, 2)
    see = _visible(s, n)[:, None, :, None]                                # [B][1][T][1][n]
    q = s["q"].float().reshape(c["b"], c["t"], c["hkv"], -1, c["d"]).permute(0, 2, 1, 3, 4)
    grp = q.shape[3]
    k = _values(s, "k", slots)
    x = (q.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (c["t"], grp)) / math.sqrt(c["d"])
    del k
    x = torch.where(see, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.where(see, torch.exp(x - torch.where(m == -math.inf, 0.0, m)), 0.0)
    del x
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ _values(s, "v", slots)).unflatten(2, (c["t"], grp))
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(s["out"].shape)
    live = torch.arange(c["t"], device=DEV) < s["count"][:, None]
    s["out"].copy_(torch.where(live[..., None, None], o.to(s["out"].dtype), s["out"]))
    return s["out"]


def _plain_commit(s):
    c = s["case"]
    i = torch.arange(c["t"], device=DEV)
    live = i < s["n_accept"][:, None]
    past = s["n_past"][:, None].long()
    src = _slots(s, torch.where(live, past + s["path"], 0))[live]
    dst = _slots(s, torch.where(live, past + i, 0))[live]
    for key in ("k", "v"):
        _flat(s, key)[dst] = _flat(s, key)[src]
        if key + "_scale" in s:
            s[key + "_scale"].view(-1)[dst] = s[key + "_scale"].view(-1)[src]
    return {k: s[k] for k in ("k", "v", "k_scale", "v_scale") if k in s}


def _own(s):
    from autoregressive_codebook_tts_gb300 import tts
    c = s["case"]
    if c["op"] == "rope":
        qd, kd = c["hq"] * c["d"], c["hkv"] * c["d"]
        if "q_out" not in s:
            s["q_out"] = torch.empty(c["rows"], qd, dtype=DT[c["out_dtype"]], device=DEV)
            s["k_out"] = torch.empty(c["rows"], kd, dtype=DT[c["out_dtype"]], device=DEV)
        tts.tts_rope_rows(s["rows"][:, :qd], s["rows"][:, qd: qd + kd], s["q_out"], s["k_out"], s["pos"], c["hq"],
                          c["hkv"], c["d"], s["cs"], gamma_q=s["gq"] if c["norm"] else None,
                          gamma_k=s["gk"] if c["norm"] else None, eps=1e-6, interleaved=c["inter"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "table":
        cs = torch.empty(c["max_pos"], c["rot"] // 2, 2, device=DEV)
        tts.tts_rope_table_scaled(cs, c["max_pos"], c["rot"], s["base"], kind=c["kind"], factor=c["factor"],
                                  original_max_pos=c["original"], low_rotations=1.0, high_rotations=32.0,
                                  attn_scale=c["attn_scale"])
        return cs
    if "desc" not in s:
        s["desc"] = tts.kv_desc(c["b"], c.get("hq", c["hkv"]), c["hkv"], c["d"], _capacity(c), c["kv"],
                                paged=c["page"] > 0, page_size=c["page"], n_pages=s["pages"],
                                block_table=s.get("table"))
        s["cache"] = tts.kv_cache(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))
    if c["op"] == "kv":
        kd = c["hkv"] * c["d"]
        tts.tts_kv_write_rows(s["src"][:, :kd], s["src"][:, kd:], s["cache"], s["desc"], s["n_past"], c["t"],
                              n_rows=s["count"] if c["ragged"] else None)
        n = s["k_out"].shape[1]
        if c["window"]:
            if "zero" not in s:
                s["zero"] = torch.zeros_like(s["n_past"])
            tts.tts_kv_read_rows(s["cache"], s["desc"], s["zero"], n, s["k_out"].view(-1, kd), s["v_out"].view(-1, kd),
                                 n_rows=s["n_past"] + s["count"])
        else:
            tts.tts_kv_read_rows(s["cache"], s["desc"], s["n_past"], n, s["k_out"].view(-1, kd), s["v_out"].view(-1, kd),
                                 n_rows=s["count"] if c["ragged"] else None)
        got = {"k": s["k_out"], "v": s["v_out"]}
        return dict(got, ks=s["k_scale"], vs=s["v_scale"]) if c["kv"] in TOP else got
    if c["op"] == "tree":
        if "ws" not in s:
            s["ws"] = tts.tree_workspace(s["desc"], c["t"], q_dtype=c["q"])
        tts.tts_tree_attn(s["q"].view(c["b"] * c["t"], -1), s["cache"], s["desc"], s["n_past"], c["t"],
                          1.0 / math.sqrt(c["d"]), s["out"], s["ws"], n_nodes=s["count"] if c["ragged"] else None,
                          tree_mask=s["mask"])
        return s["out"]
    tts.tts_tree_commit(s["cache"], s["desc"], s["n_past"], s["path"], s["n_accept"], c["t"])
    return {k: s[k] for k in ("k", "v", "k_scale", "v_scale") if k in s}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, stream by stream
# ---------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    return {"rope": _exact_rope, "table": _exact_table, "kv": _exact_kv, "tree": _exact_tree,
            "commit": _exact_commit}[c["op"]](c, s)


def _exact_rope(c, s):
    x = s["rows"].double().view(c["rows"], -1, c["d"])
    cs = torch.view_as_complex(s["cs"].double())[s["pos"].long()]
    half, out = c["rot"] // 2, {}
    for key, lo, h, gam in (("q", 0, c["hq"], s["gq"]), ("k", c["hq"], c["hkv"], s["gk"])):
        y = x[:, lo: lo + h].clone()
        if c["norm"]:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["d"] + 1e-6) * gam.double()
        first = torch.arange(half, device=DEV) * 2 if c["inter"] else torch.arange(half, device=DEV)
        second = first + 1 if c["inter"] else first + half
        z = torch.complex(y[..., first], y[..., second]) * cs[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        out[key] = y.reshape(c["rows"], h * c["d"])
    return out


def _exact_table(c, s):
    d, f = c["rot"], []
    for i in range(d // 2):
        b = s["base"] * (c["factor"] ** (d / (d - 2.0)) if c["kind"] == "base" else 1.0)
        w = b ** (-2.0 * i / d)
        if c["kind"] == "linear":
            w /= c["factor"]
        if c["kind"] == "parts":
            turns = c["original"] / (2 * math.pi / w)
            keep = 0.0 if turns < 1 else 1.0 if turns > 32 else (turns - 1.0) / 31.0
            w = (1 - keep) * w / c["factor"] + keep * w
        f.append(w)
    a = np.outer(np.arange(c["max_pos"], dtype=np.float64), np.array(f))
    return torch.from_numpy(np.stack([np.cos(a), np.sin(a)], -1) * c["attn_scale"])


def _row_at(c, s, b, pos):
    """(first index, second index) of positions pos of stream b in [n][Hkv][rows]."""
    if not c["page"]:
        return torch.full_like(pos, b), pos
    return s["table"][b].long()[pos // c["page"]], pos % c["page"]


_E4M3 = sorted({(m / 8 + (e > 0)) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8) if (e, m) != (15, 7)})


def _nearest(x, kv):
    """The nearest code by search among all of them; a tie goes to the even one."""
    codes = _E4M3 if kv == "e4m3" else [float(i) for i in range(128)]
    grid = torch.tensor(codes, device=DEV, dtype=torch.float64)
    mid = (grid[1:] + grid[:-1]) / 2
    a = x.abs()
    low, high = torch.searchsorted(mid, a), torch.searchsorted(mid, a, right=True)
    i = torch.where((low != high) & (low % 2 == 1), high, low)
    return torch.sign(x) * grid[i]


def _cast(t):
    return t.double() if t.dtype != torch.float8_e4m3fn else t.float().double()


def _exact_kv(c, s):
    lens, counts = _lens(c), _counts(c)
    src = s["src"].double().view(c["b"], c["t"], 2, c["hkv"], c["d"])
    g = torch.arange(c["hkv"], device=DEV)
    outs = {"k": s["k_out"].double(), "v": s["v_out"].double()}
    for i, key in enumerate(("k", "v")):
        for b in range(c["b"]):
            pos = torch.arange(lens[b], lens[b] + counts[b], device=DEV)
            at, row = _row_at(c, s, b, pos)
            x = src[b, : counts[b], i]
            if c["kv"] in TOP:
                sc = (x.abs().amax(-1) / TOP[c["kv"]]).float()
                new = _nearest(x / sc[..., None].double(), c["kv"]) * sc[..., None].double()
                s[key + "_scale"][at[:, None], g, row[:, None]] = sc
            else:
                new = x.to(CACHE_DT[c["kv"]]).double()
            if c["window"]:
                at, row = _row_at(c, s, b, torch.arange(lens[b], device=DEV))
                raw = s[key].view(torch.uint8) if c["kv"] == "e4m3" else s[key]
                old = raw[at[:, None], g, row[:, None]]
                old = _cast(old.view(torch.float8_e4m3fn) if c["kv"] == "e4m3" else old)
                if c["kv"] in TOP:
                    old = old * s[key + "_scale"][at[:, None], g, row[:, None]][..., None].double()
                new = torch.cat([old, new])
            outs[key][b, : new.shape[0]] = new
    return dict(outs, ks=s["k_scale"].double(), vs=s["v_scale"].double()) if c["kv"] in TOP else outs


def _exact_tree(c, s):
    lens, counts = _lens(c), _counts(c)
    out = s["out"].double()
    g = torch.arange(c["hkv"], device=DEV)
    for b in range(c["b"]):
        n, k = lens[b], counts[b]
        at, row = _row_at(c, s, b, torch.arange(n + k, device=DEV))
        kv = []
        for key in ("k", "v"):
            raw = s[key].view(torch.uint8) if c["kv"] == "e4m3" else s[key]
            x = raw[at[:, None], g, row[:, None]]
            x = _cast(x.view(torch.float8_e4m3fn) if c["kv"] == "e4m3" else x)
            if c["kv"] in TOP:
                x = x * s[key + "_scale"][at[:, None], g, row[:, None]][..., None].double()
            kv.append(x.repeat_interleave(c["hq"] // c["hkv"], 1))        # [n + k][Hq][D]
        x = torch.einsum("thd,nhd->htn", s["q"][b, :k].double(), kv[0]) * c["d"] ** -0.5
        bits = None if s["mask"] is None else s["mask"][b, :k].cpu().tolist()
        see = torch.zeros(k, n + k, dtype=torch.bool)
        see[:, :n] = True
        for t in range(k):
            for u in range(k):
                see[t, n + u] = u <= t if bits is None else bool(bits[t] >> u & 1)
        x = x.masked_fill(~see.to(DEV), -math.inf)
        out[b, :k] = torch.einsum("htn,nhd->thd", torch.softmax(x, -1), kv[1])
    return out


def _exact_commit(c, s):
    n_past, path, n = s["n_past"].cpu().tolist(), s["path"].cpu().tolist(), s["n_accept"].cpu().tolist()
    keys = [k for k in ("k", "v", "k_scale", "v_scale") if k in s]
    for b in range(c["b"]):
        for i in range(n[b]):
            pos = torch.tensor([n_past[b] + path[b][i], n_past[b] + i], device=DEV)
            at, row = (x.tolist() for x in _row_at(c, s, b, pos))
            for k in keys:
                s[k][at[1], :, row[1]] = s[k][at[0], :, row[0]]
    return {k: s[k] if s[k].dtype == torch.int8 else s[k].double() for k in keys}
