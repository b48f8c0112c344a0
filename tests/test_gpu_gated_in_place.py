"""The gradients of gate and up in place of them, as the header allows, in every kind of tile."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests import test_gpu_gated as gated
from tests.block_helpers import BF16, FP16, padding_kept, strided
from tests.test_gpu_largest_tiles import largest_of
from tests.test_gpu_wide_tiles import EDGES

pytestmark = pytest.mark.gpu
IN_PLACE = {"64x16": ([30, 9], 72, 264), "128x16": ([0, 1, 2, 5] * 75, 264, 272), "128x64": ([30, 1, 64, 0, 17, 65, 32, 31] * 5, 520, 528),
            "128x128": ([500, 129, 0, 900, 640, 831], 1288, 264), "largest": (EDGES, 2568, 256)}


@pytest.mark.parametrize("tile", IN_PLACE)
@pytest.mark.parametrize("odd", [0, 1], ids=["aligned", "unaligned"])
def test_gradients_in_place(tile, odd):
    """The same bits as beside them, and gates' rows at odd addresses do not change them either."""
    sizes, n, k = IN_PLACE[tile]
    n += odd and 1
    if tile == "largest" and not odd:
        largest_of("hidden", sizes, n, k, before=5, after=3)
    s = gated.make(sizes, n, k, (BF16, FP16)[odd], seed=47, before=5, after=3, act=("silu", "gelu")[odd])
    want = gated.check_hidden(s)
    for a, b in zip(gated.check_hidden(s, in_place=True), want):
        assert torch.equal(a, b)
    plan = R.Gated(s["groups"], n, k, s["t"], act=s["act"], limit=s["limit"], gate_stride=n + 3)
    (gate, kept), (up, beside) = (strided(s["rows"], n, s["t"], 3, 1) for _ in range(2))
    gate.copy_(s["gate"])
    up.copy_(s["up"])
    h = torch.empty_like(want[2])
    R.gated_backward_h(plan, s["dy"], s["w_down"], gate, up, s["off"], gate, up, h)
    for a, b in zip((gate, up, h), want):
        assert torch.equal(a, b)
    assert padding_kept(gate, kept) and padding_kept(up, beside)
