"""Numerics of the drafted-decoding calls at the far ends of their ranges.  References and bounds
as in test_draft_gpu.
"""
import numpy as np
import pytest
import torch

import draft_ref as R
from test_draft_gpu import ints, tts  # noqa: F401

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
