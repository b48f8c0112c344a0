"""The example block: its training step against the formulas in 64 bits, and its decode step.

Tolerances. The example rounds to 16 bits between its operators: rows' products
(a, d), silu, the block's output and the gradients between them, a handful of
half steps of 2^-8 (bf16) or 2^-11 (fp16) each in relative terms of what they
enter. Errors of different elements are independent, so norms over whole
tensors are compared: a chain of at most 8 roundings stays below 8 half steps of the norm."""
import pytest
import torch

from examples.block_step import Block, Decode, inputs
from tests.block_helpers import BF16, F32, FP16, half_step

pytestmark = pytest.mark.gpu


def near(got, want, dtype, what):
    off = float((got.double() - want).norm() / want.norm())
    assert off <= 8 * half_step(dtype), f"{what}: {off:.3g}"


def reference(block, x, y, picks, weights, shared=None):
    """x', y' and the block's output by autograd in 64 bits, weights as leaves."""
    leaves = {k: getattr(block, k).double().requires_grad_() for k in ("w_up", "w_down", "w_post", "w_pre", "gate")}
    leaves["x"], leaves["y"] = x.double().requires_grad_(), y.double().requires_grad_()
    b = torch.zeros_like(leaves["y"])
    for e in range(block.experts):
        token, pick = (picks == e).nonzero(as_tuple=True)
        if token.numel():
            h = torch.nn.functional.silu(leaves["y"][token] @ leaves["w_up"][e].t())
            b = b.index_add(0, token, (h @ leaves["w_down"][e].t()) * weights.double()[token, pick][:, None])
    if shared is not None:
        b = b + shared
    eps, scale = block.join.eps, block.join.scale

    def norm(v):
        return v * (v.pow(2).mean(-1, keepdim=True) + eps).rsqrt()

    x_out = leaves["x"] + scale * leaves["gate"] * norm(b) * leaves["w_post"]
    return x_out, norm(x_out) * leaves["w_pre"], leaves


@pytest.mark.parametrize("dtype,residual", [(BF16, BF16), (FP16, F32)], ids=["bf16", "fp16-f32"])
def test_training_step(dtype, residual):
    block = Block(dim=264, inter=136, experts=7, topk=3, tokens=90, dtype=dtype, residual=residual)
    x, y, picks, weights = inputs(block, 90)
    picks = picks % 6   # an expert without rows
    x_out, y_out, kept = block.forward(x, y, picks, weights)
    gen = torch.Generator(device="cuda").manual_seed(3)
    dy, dx_out = torch.randn(y.shape, generator=gen, device="cuda").to(dtype), torch.randn(x.shape, generator=gen, device="cuda").to(x.dtype)
    dx, dyin, grads = block.backward(dy, dx_out, kept)
    wx, wy, leaves = reference(block, x, y, picks, weights)
    near(x_out, wx.detach(), dtype, "x'")
    near(y_out, wy.detach(), dtype, "y'")
    ((wy * dy.double()).sum() + (wx * dx_out.double()).sum()).backward()
    near(dx, leaves["x"].grad, dtype, "dx")
    near(dyin, leaves["y"].grad, dtype, "dy")
    for k, g in grads.items():
        near(g, leaves[k].grad, dtype, k)
    assert not grads["w_up"][6].any() and not grads["w_down"][6].any()


@pytest.mark.parametrize("tokens", [1, 30])
def test_decode_step(tokens):
    block = Block(dim=264, inter=136, experts=7, topk=3, tokens=90)
    decode = Decode(block, adapters=4, rank=8, tokens=90)
    x, y, picks, weights = inputs(block, tokens, seed=2)
    request = torch.arange(tokens, dtype=torch.int32, device="cuda") % 5 - 1
    shared = y.double() @ decode.w.double().t()
    for t in range(tokens):
        i = int(request[t])
        if i >= 0:
            shared[t] += float(decode.factor[i]) * (decode.b[i].double() @ (decode.a[i].double() @ y[t].double()))
    wx, wy, _ = reference(block, x, y, picks, weights, shared)
    near(decode.step(x, y, picks, weights, request), wy.detach(), BF16, "y'")
    near(x, wx.detach(), BF16, "x'")
