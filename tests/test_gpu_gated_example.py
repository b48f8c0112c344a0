"""The example's gated block: its training step against the formulas in 64 bits, and its 4-bit form step by step.

Tolerances as for the example's other block: at most 8 roundings of half a step in a chain, norms over whole tensors."""
import pytest
import torch

from examples.block_step import Decode, FourBitBlock, GatedBlock, inputs
from tests.block_helpers import BF16, F32, FP16
from tests.gated_helpers import hidden
from tests.mx_helpers import quantised, values
from tests.test_gpu_block_example import near

pytestmark = pytest.mark.gpu
SIZES = dict(dim=264, inter=136, experts=7, topk=3, tokens=90)


@pytest.mark.parametrize("dtype,residual", [(BF16, BF16), (FP16, F32)], ids=["bf16", "fp16-f32"])
def test_training_step(dtype, residual):
    block = GatedBlock(**SIZES, dtype=dtype, residual=residual)
    x, y, picks, weights = inputs(block, 90)
    picks = picks % 6   # an expert without rows
    x_out, y_out, kept = block.forward(x, y, picks, weights)
    gen = torch.Generator(device="cuda").manual_seed(3)
    dy, dx_out = torch.randn(y.shape, generator=gen, device="cuda").to(dtype), torch.randn(x.shape, generator=gen, device="cuda").to(x.dtype)
    dx, dyin, grads = block.backward(dy, dx_out, kept)

    names = ("w_gate", "w_up", "w_down", "w_post", "w_pre", "gate")
    leaves = {k: getattr(block, k).double().requires_grad_() for k in names}
    wx, wy = x.double().requires_grad_(), y.double().requires_grad_()
    b = torch.zeros_like(wy)
    for e in range(block.experts):
        token, pick = (picks == e).nonzero(as_tuple=True)
        if token.numel():
            h = hidden(wy[token] @ leaves["w_gate"][e].t(), wy[token] @ leaves["w_up"][e].t(), "silu", 7.0)
            b = b.index_add(0, token, (h @ leaves["w_down"][e].t()) * weights.double()[token, pick][:, None])

    def norm(v):
        return v * (v.pow(2).mean(-1, keepdim=True) + block.join.eps).rsqrt()

    out = wx + block.join.scale * leaves["gate"] * norm(b) * leaves["w_post"]
    normed = norm(out) * leaves["w_pre"]
    near(x_out, out.detach(), dtype, "x'")
    near(y_out, normed.detach(), dtype, "y'")
    ((normed * dy.double()).sum() + (out * dx_out.double()).sum()).backward()
    near(dx, wx.grad, dtype, "dx")
    near(dyin, wy.grad, dtype, "dy")
    for k, g in grads.items():
        near(g, leaves[k].grad, dtype, k)
    assert set(grads) == set(names) and not any(grads[k][6].any() for k in ("w_gate", "w_up", "w_down"))


@pytest.mark.parametrize("tokens", [1, 30])
def test_in_4_bits(tokens):
    block = FourBitBlock(**SIZES)
    decode = Decode(block, adapters=4, rank=8, tokens=90)
    x, y, picks, weights = inputs(block, tokens, seed=2)
    _, (order, ends, rows, row, h, four) = block.experts_forward(y, picks, weights)
    d, _ = block.rows_forward(rows, ends)

    def same(v, got):
        for a, b in zip(quantised(v.cpu().flatten(0, -2), "ceil"), got):
            assert torch.equal(a, b.cpu().flatten(0, -2))
        return values(*got, v.shape[-1])

    qx, qh = same(rows, row), same(h, four)
    w_gate, w_up, w_down = (same(w, q) for w, q in ((block.w_gate, block.four_gate), (block.w_up, block.four_up),
                                                    (block.w_down, block.four_down)))
    expert = picks.flatten()[order]
    for e in expert.unique().tolist():
        m = expert == e
        near(h[m], hidden(qx[m] @ w_gate[e].t(), qx[m] @ w_up[e].t(), "silu", 7.0), BF16, "h")
        near(d[m], qh[m] @ w_down[e].t(), BF16, "d")
    request = torch.arange(tokens, dtype=torch.int32, device="cuda") % 5 - 1
    assert decode.step(x, y, picks, weights, request).isfinite().all()
