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
