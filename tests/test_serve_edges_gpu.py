"""Inputs of the calls that serve many requests at once that the contract allows and that are easily
missed: adapters named by any negative number, on each of the projection's kernels.

Tolerances are those of test_serve_gpu (check_project); what is compared with equality is exact
in f32.
"""
import pytest
import torch

import serve_ref as R
from test_serve_gpu import I32, check_project, flag, gen, ints, project_case, randn, run_project, tts  # noqa: F401

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
