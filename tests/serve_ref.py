"""Plain restatements, in 64 bits or whole numbers, of the calls that serve many requests at once
(tts_add_rms_norm, tts_project_rows, tts_page_plan).  Written from the formulas of
include/tts_decode.h; shares no code with the library."""
import numpy as np
import torch

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
# half a step of a type, relative to the value
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}


def norm(x, res, gamma, eps, res_dtype):
    """(h, y): the stored sum and the normed row, float64."""
    h = x.double()
    if res is not None:
        h = (res.float() + x.float()).to(res_dtype).double()
    return h, h * (h.square().mean(-1, keepdim=True) + eps) ** -0.5 * gamma.double()


_GRID = torch.tensor(sorted({(m / 8 + (e > 0)) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)
                             if (e, m) != (15, 7)}), dtype=torch.float64)


def e4m3(x):
    """The nearest code to each float64 value, a tie to the even one; codes as float64."""
    grid = _GRID.to(x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    a = x.abs()
    low, high = torch.searchsorted(mid, a), torch.searchsorted(mid, a, right=True)
    i = torch.where((low != high) & (low % 2 == 1), high, low)
    return torch.where(x < 0, -1.0, 1.0) * grid[i]


def project(x, w, a, b, rank, scale, adapter, x_scale=None, w_scale=None):
    """(y, mass): the rows in float64 (adapter[r] < 0: none), and the sums of magnitudes that
    rounding errors of the sums are relative to: K and adapter parts."""
    x, w = x.float().double(), w.float().double()
    if x_scale is not None:
        x, w = x * x_scale.double()[:, None], w * w_scale.double()[:, None]
    y, mass = x @ w.T, x.abs() @ w.abs().T
    if a is not None:
        for i in sorted({int(i) for i in adapter.tolist() if i >= 0}):
            at = (adapter == i).nonzero()[:, 0]
            r = int(rank[i])
            ai, bi = a[i, :r].double(), b[i, :, :r].double()
            v = x[at] @ ai.T
            y[at] += float(scale[i]) * (v @ bi.T)
            mass[at] += abs(float(scale[i])) * ((x[at].abs() @ ai.abs().T) @ bi.abs().T)
    return y, mass


def plan(table, free, n_free, n_past, n_new, n_pages, page, capacity, max_rows, T):
    """One step in plain Python: the new table, list, count, and the maps; whether each kind of
    refusal happened."""
    table, free = [list(map(int, r)) for r in table], list(map(int, free))
    B = len(table)
    flags = set()
    if not 0 <= n_free <= n_pages:
        flags.add("nvalid")
    stack = free[:min(max(n_free, 0), n_pages)]
    held = lambda i: 0 <= i < n_pages  # noqa: E731
    lost = False
    for b in range(B):
        if n_new[b] < 0:
            for i in range(capacity // page):
                if held(table[b][i]):
                    if len(stack) < n_pages:
                        stack.append(table[b][i])
                    else:
                        lost = True
                    table[b][i] = -1
    if lost:
        flags.add("page")
    after = stack + free[len(stack):]
    out_of_pages, sum_need, sum_rows = len(stack), 0, 0
    n_rows, used = [0] * B, 0
    for b in range(B):
        n, p = n_new[b], n_past[b]
        if n <= 0:
            continue
        if p < 0 or p + n > capacity or (T > 0 and n > T):
            flags.add("nvalid")
            continue
        want = [i for i in range(p // page, (p + n - 1) // page + 1) if not held(table[b][i])]
        sum_need += len(want)
        if want and sum_need > out_of_pages:
            flags.add("page")
            continue
        sum_rows += n
        if T == 0 and sum_rows > max_rows:
            flags.add("nvalid")
            continue
        n_rows[b] = n
        for i in want:
            table[b][i] = stack[len(stack) - 1 - used]
            used += 1
    start = [0]
    for b in range(B):
        start.append(start[-1] + (T if T > 0 else n_rows[b]))
    stream, pos, slot = [-1] * max_rows, [0] * max_rows, [-1] * max_rows
    for b in range(B):
        for t in range(n_rows[b]):
            r, q = start[b] + t, n_past[b] + t
            stream[r], pos[r] = b, q
            g = table[b][q // page]
            if held(g):
                slot[r] = g * page + q % page
            else:
                flags.add("page")
    return {"table": np.array(table), "free": np.array(after), "n_free": len(stack) - used, "n_rows": n_rows,
            "row_start": start, "row_stream": stream, "row_pos": pos, "row_slot": slot, "flags": flags}
