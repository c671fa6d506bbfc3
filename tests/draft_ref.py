"""Plain 64-bit restatements of the drafted-decoding calls (CPU, loops where loops are the
definition), and the inputs of their tests."""
import math

import numpy as np
import torch

TOP = {"i8": 127.0, "e4m3": 448.0}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}
# every finite magnitude of a 4-exponent-bit, 3-mantissa-bit number (bias 7, no infinities)
E4M3 = np.array(sorted({(m / 8 + (e > 0)) * 2.0 ** (max(e, 1) - 7)
                        for e in range(16) for m in range(8) if (e, m) != (15, 7)}))


def nearest_code(x, kv):
    """The code values nearest to x (f64 quotients), ties to the even code, at most TOP."""
    grid = E4M3 if kv == "e4m3" else np.arange(128.0)
    a = np.minimum(np.abs(x), TOP[kv])
    hi = np.clip(np.searchsorted(grid, a), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return np.copysign(np.where(take_hi, grid[hi], grid[lo]), x)


def quantise(x, kv):
    """(code values, scales) of rows x [..., D] f32: the definition in the header."""
    x = np.asarray(x, np.float32)
    top = np.abs(x).max(-1)
    bad = ~np.isfinite(x).all(-1)
    with np.errstate(all="ignore"):
        s = top * (np.float32(1) / np.float32(TOP[kv]))
        s[bad] = np.nan
        zero = bad | (s == 0)
        q = x.astype(np.float64) / np.where(zero, 1.0, s.astype(np.float64))[..., None]
        q = np.where(zero[..., None], 0.0, q)
    return nearest_code(q, kv), s


def to_cache(x, kv):
    """f32 rows as (cache tensor of codes or entries, scales or None)."""
    x = np.asarray(x, np.float32)
    if kv in TOP:
        c, s = quantise(x, kv)
        return torch.from_numpy(c).to(torch.float32).to(TORCH[kv]), torch.from_numpy(s)
    return torch.from_numpy(x).to(TORCH[kv]), None


def values(t, s):
    """A cache tensor as f64 values."""
    v = t.float().double()
    return v if s is None else v * s.double()[..., None]


class Cache:
    """A random cache on the device with a host copy; every slot outside the streams' windows
    is NaN (f32, bf16) or carries a NaN scale (8-bit)."""

    def __init__(self, B, hkv, d, capacity, kv, page=0, seed=0, extra_pages=3, fill=None, std=1.0):
        g = np.random.default_rng(seed)
        self.B, self.hkv, self.d, self.cap, self.kv, self.page = B, hkv, d, capacity, kv, page
        if page:
            per = capacity // page
            self.n_pages = B * per + extra_pages
            self.bt = torch.from_numpy(g.permutation(self.n_pages)[: B * per].reshape(B, per).astype(np.int32))
            shape = (self.n_pages, hkv, page, d)
        else:
            self.n_pages, self.bt = 0, None
            shape = (B, hkv, capacity, d)
        self.k, self.ks = to_cache(g.standard_normal(shape, np.float32) * std, kv)
        self.v, self.vs = to_cache(g.standard_normal(shape, np.float32) * std, kv)
        if fill is not None:
            live = torch.zeros(shape[0], shape[2], dtype=torch.bool)
            for b in range(B):
                for j in range(int(fill[b])):
                    at, row = self.at(b, j)
                    live[at, row] = True
            dead = ~live[:, None, :].expand(shape[:-1])
            for t, s in ((self.k, self.ks), (self.v, self.vs)):
                if s is None:
                    t[dead] = float("nan")
                else:
                    s[dead] = float("nan")

    def at(self, b, j):
        return (b, j) if not self.page else (int(self.bt[b, j // self.page]), j % self.page)

    def rows(self, which, b, n):
        """f64 values of positions [0, n) of stream b: [n, hkv, d]."""
        t, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        out = torch.empty(n, self.hkv, self.d, dtype=torch.float64)
        for j in range(n):
            at, row = self.at(b, j)
            out[j] = values(t[at, :, row].clone(), None if s is None else s[at, :, row])
        return out

    def to_device(self, tts, hq, dev="cuda"):
        self.dk, self.dv = self.k.to(dev), self.v.to(dev)
        self.dks = None if self.ks is None else self.ks.to(dev)
        self.dvs = None if self.vs is None else self.vs.to(dev)
        self.dbt = None if self.bt is None else self.bt.to(dev)
        self.desc = tts.kv_desc(self.B, hq, self.hkv, self.d, self.cap, self.kv, window_quantum=1,
                                paged=self.page > 0, page_size=self.page, n_pages=self.n_pages,
                                block_table=self.dbt)
        self.cache = tts.kv_cache(self.dk, self.dv, self.dks, self.dvs)
        return self

    def back(self):
        """The device tensors (K, V, scales) on the host, as bytes."""
        ts = [self.dk, self.dv] + ([self.dks, self.dvs] if self.dks is not None else [])
        return [t.cpu().contiguous().view(torch.uint8) for t in ts]

    def host(self):
        ts = [self.k, self.v] + ([self.ks, self.vs] if self.ks is not None else [])
        return [t.contiguous().view(torch.uint8) for t in ts]


def random_tree(T, rng, empty=0.0):
    """T nodes' ancestor bits (with the node's own) as int64; some nodes see nothing."""
    m = [0] * T
    for t in range(T):
        up = m[rng.integers(0, t)] if t and rng.random() < 0.85 else 0
        m[t] = up | (1 << t)
    m = [0 if rng.random() < empty else x for x in m]
    return np.array(m, np.uint64).view(np.int64)


def tree_attn(cache, q, past, nodes, mask, scale):
    """q [B, T, Hq, D] f64 -> (out, mean |v| under the weights), rows past the nodes NaN.
    mask int64 [B, T] or None (the chain)."""
    B, T, Hq, D = q.shape
    out = torch.full((B, T, Hq, D), float("nan"), dtype=torch.float64)
    mag = torch.full_like(out, float("nan"))
    grp = Hq // cache.hkv
    for b in range(B):
        n = past[b] + nodes[b]
        if nodes[b] == 0:
            continue
        K, V = cache.rows("k", b, n), cache.rows("v", b, n)
        for t in range(nodes[b]):
            bits = (2 << t) - 1 if mask is None else int(mask[b][t]) & ((1 << 64) - 1)
            see = [j for j in range(n) if j < past[b] or (bits >> (j - past[b])) & 1]
            if not see:
                out[b, t] = 0
                mag[b, t] = 0
                continue
            k = K[see].repeat_interleave(grp, 1)
            v = V[see].repeat_interleave(grp, 1)
            w = torch.softmax(torch.einsum("hd,nhd->hn", q[b, t], k) * scale, -1)
            out[b, t] = torch.einsum("hn,nhd->hd", w, v)
            mag[b, t] = torch.einsum("hn,nhd->hd", w, v.abs())
    return out, mag


def rope(x, pos, cs, rot, inter, gamma=None, eps=1e-6):
    """x [rows, heads, D] f64; cs [max_pos, rot / 2, 2] f32 table."""
    x = x.clone()
    D = x.shape[-1]
    if gamma is not None:
        x = x * (x.square().mean(-1, keepdim=True) + eps) ** -0.5 * gamma.double()
    c, s = cs.double()[pos.long()][:, None].unbind(-1)
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    xa, xb = x[..., a].clone(), x[..., b].clone()
    x[..., a] = xa * c - xb * s
    x[..., b] = xa * s + xb * c
    return x


def table(max_pos, rot, base, kind="none", factor=1.0, L=1, low=1.0, high=32.0, attn=1.0):
    out = np.empty((max_pos, rot // 2, 2))
    for i in range(rot // 2):
        b = base * (factor ** (rot / (rot - 2)) if kind == "base" else 1.0)
        f = b ** (-2.0 * i / rot)
        if kind == "linear":
            f /= factor
        if kind == "parts":
            r = L * f / (2 * math.pi)
            w = min(max((r - low) / (high - low), 0.0), 1.0)
            f = f * (w + (1 - w) / factor)
        a = np.arange(max_pos, dtype=np.float64) * f
        out[:, i, 0], out[:, i, 1] = attn * np.cos(a), attn * np.sin(a)
    return out
