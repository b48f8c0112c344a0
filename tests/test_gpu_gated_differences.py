"""The gradients of gate and up against differences of what the forward call gives."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests.block_helpers import FP16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,limit", [("silu", 0.0), ("gelu", 0.0), ("silu", 2.0), ("gelu", 2.0)])
def test_gradients_against_differences(act, limit):
    """h of the forward call at g and u a step to either side, which fp16 and the products (one term each) hold exactly.

    A central difference of step d is off by d^2 / 6 of the third derivative (of act below 1.1, of the product with u: that
    times u), and by the two roundings of h: half a step of fp16 of each, over 2 d; the gradient by its own rounding. The
    clamps' corners have no slope and are left out."""
    d = 0.125
    value = torch.arange(-48, 49) * 0.0625 + 0.03125   # -2.97 to 3.03
    g, u = (v.flatten() for v in torch.meshgrid(value, value[::6], indexing="ij"))
    rows, k, n = g.numel(), 8, 8
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    plan = R.Gated(1, n, k, FP16, act=act, limit=limit)
    w_gate, w_up, w_down = (torch.zeros((1, 8, 8), dtype=FP16, device="cuda") for _ in range(3))
    w_gate[:, :, 0], w_up[:, :, 1], w_down[:, 2] = 1.0, 1.0, 1.0

    def forward(g, u):
        x = torch.zeros((rows, k), dtype=FP16, device="cuda")
        x[:, 0], x[:, 1] = g, u
        h, gate, up = (torch.empty((rows, n), dtype=FP16, device="cuda") for _ in range(3))
        R.gated_forward(plan, x, w_gate, w_up, off, h, gate, up)
        assert torch.equal(gate[:, 3].cpu(), g.half()) and torch.equal(up[:, 3].cpu(), u.half())
        return h.double().cpu()[:, 3], gate, up

    h, gate, up = forward(g, u)
    dy = torch.zeros((rows, k), dtype=FP16, device="cuda")
    dy[:, 2] = 1.0
    dgate, dup, again = (torch.empty_like(gate) for _ in range(3))
    R.gated_backward_h(plan, dy, w_down, gate, up, off, dgate, dup, again)
    assert torch.equal(again.double().cpu()[:, 3], h)
    half = 2.0 ** -11
    for got, (hi, lo), clear, third in ((dgate, (forward(g + d, u)[0], forward(g - d, u)[0]), (g - 2).abs() > d, 1.1 * u.abs()),
                                        (dup, (forward(g, u + d)[0], forward(g, u - d)[0]), (u.abs() - 2).abs() > d, 0.0 * u)):
        want, got = (hi - lo) / (2 * d), got.double().cpu()[:, 3]
        tol = d * d / 6 * third + half * (hi.abs() + lo.abs()) / (2 * d) + half * got.abs() + 2.0 ** -17 * (1 + u.abs()) / d
        keep = clear if limit else torch.ones_like(clear)
        off_by = ((got - want).abs() - tol)[keep]
        assert off_by.max() <= 0, float(off_by.max())
