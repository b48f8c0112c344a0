"""The activation's gradients at gates up to the largest finite ones, where the polynomial of gelu's derivative leaves the
range of f32 long after its factor 1 - s has become 0: the derivative there is 1, and 0 at the other end.

Tolerances: the activation's own errors of gated_helpers and one rounding to bf16. h's gradient is 1, exactly: one term."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests.block_helpers import BF16, assert_within
from tests.gated_helpers import ACT, SLOPE, gradients, hidden
from tests.test_gpu_gated import rounded
from tests.test_gpu_wide_tiles import EDGES

pytestmark = pytest.mark.gpu
GATES = [1e2, 103.0, 104.0, 105.0, 1e3, 1e6, 1e12, 1.8e19, 1.9e19, 1e20, 1e25, 1e30, 3e38, float(torch.finfo(BF16).max)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("limit", [0.0, 1e30], ids=["no limit", "a large limit"])
@pytest.mark.parametrize("sizes,n,k", [([28, 0, 28], 8, 8), ([28, 0, 28], 9, 7), (EDGES, 2568, 256)],
                         ids=["small", "unaligned", "largest tiles"])
def test_finite_gates(sizes, n, k, limit, act):
    rows, groups = sum(sizes), len(sizes)
    off = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    values = torch.tensor(GATES + [-v for v in GATES]).to(BF16).cuda()
    at = torch.arange(rows, device="cuda")[:, None] + 3 * torch.arange(n, device="cuda")
    gate = values[at % values.numel()]
    up = torch.where(at // values.numel() % 2 == 0, 0.75, -1.5).to(BF16)   # (products of 1.5 and the largest gate: dup's alone)
    dy = torch.zeros((rows, k), dtype=BF16, device="cuda")
    w_down = torch.zeros((groups, k, n), dtype=BF16, device="cuda")
    dy[:, 0], w_down[:, 0] = 1.0, 1.0
    dgate, dup, h = (torch.empty_like(gate) for _ in range(3))
    R.gated_backward_h(R.Gated(groups, n, k, BF16, act=act, limit=limit), dy, w_down, gate, up, off, dgate, dup, h)
    g, u = gate.double(), up.double()
    wg, wu = gradients(g, u, torch.ones_like(g), act, limit)
    assert_within(dgate, wg, rounded(wg, BF16) + SLOPE * u.abs() * 1.01, "dgate")
    assert_within(dup, wu, rounded(wu, BF16) + ACT * g.abs() * 1.01, "dup")
    wh = hidden(g, u, act, limit)
    inside = wh.abs() < torch.finfo(BF16).max
    assert_within(h[inside], wh[inside], rounded(wh[inside], BF16) + ACT * (g * u).abs()[inside] * 1.01, "h")
    assert not h.isnan().any()
