"""Grouped products of no rows: the status word speaks for the offsets all the same."""
import pytest
import torch

import routing_quant_expert_amd as R

pytestmark = pytest.mark.gpu

CALLS = {"forward": R.grouped_forward, "dx": R.grouped_backward_x, "dw": R.grouped_backward_w}


@pytest.mark.parametrize("way", CALLS)
@pytest.mark.parametrize("groups", [1, 2, 300])
def test_offsets_of_no_rows(way, groups):
    n, k = 64, 72
    p = R.Grouped(groups, n, k, torch.bfloat16)
    x, dy, w = (torch.zeros(v, dtype=torch.bfloat16, device="cuda") for v in ((0, k), (0, n), (groups, n, k)))
    a, b, shape = {"forward": (x, w, (0, n)), "dx": (dy, w, (0, k)), "dw": (dy, x, (groups, n, k))}[way]
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    good = [0] * (groups + 1)
    for ends, said in ((good, 0), (good[:-1] + [3], R.MOE_STATUS_BAD_OFFSETS), ([-1] + good[1:], R.MOE_STATUS_BAD_OFFSETS),
                       ([4] * (groups + 1), R.MOE_STATUS_BAD_OFFSETS)):
        off = torch.tensor(ends, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        CALLS[way](p, a, b, off, out, status)
        torch.cuda.synchronize()
        assert int(status) == said, (way, ends[:3])
