"""The operators beside the layer as a model runs them together: a training step
and a decode step of one block with experts on 16-bit weights.

    y            the normed residual stream
    rows         y's rows, one per (token, pick), sorted by expert
    h, d         h = silu(W_up[e] row), d = W_down[e] h        grouped products
    shared       W y + factor B (A y) of the token's request     adapter projection (decode)
    b            the block's output: the picks' weighted sum (+ shared)
    x', y'       the next stream and its norm                   block join

    python examples/block_step.py          # prints the step times (needs the GPU)
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import routing_quant_expert_amd as R  # noqa: E402


class Block:
    """Weights, plans and buffers that a program keeps."""

    def __init__(self, dim, inter, experts, topk, tokens, dtype=torch.bfloat16, residual=None, scale=0.7, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, sigma=1.0, mean=0.0):
            return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(sigma).add_(mean).to(dtype)

        self.dim, self.inter, self.experts, self.topk, self.dtype = dim, inter, experts, topk, dtype
        self.w_up, self.w_down = normal(experts, inter, dim, sigma=dim ** -0.5), normal(experts, dim, inter, sigma=inter ** -0.5)
        self.w_post, self.w_pre = normal(dim, sigma=0.2, mean=1.0), normal(dim, sigma=0.2, mean=1.0)
        self.gate = normal(dim, sigma=0.3, mean=0.5)
        self.join = R.Join(dim, dtype, residual=residual, scale=scale)
        self.up, self.down = R.Grouped(experts, inter, dim, dtype), R.Grouped(experts, dim, inter, dtype)
        self.up_dw = R.Grouped(experts, inter, dim, dtype, out=torch.float32)
        self.down_dw = R.Grouped(experts, dim, inter, dtype, out=torch.float32)
        self.join_ws = torch.empty(R.join_workspace_bytes(self.join, tokens), dtype=torch.uint8, device="cuda")

    def route(self, picks):
        """picks [tokens, topk] -> the sorted rows' (token, pick) places and the groups' offsets, all on the device."""
        order = picks.flatten().argsort(stable=True)
        ends = torch.zeros(self.experts + 1, dtype=torch.int32, device="cuda")
        ends[1:] = torch.bincount(picks.flatten(), minlength=self.experts).cumsum(0)
        return order, ends

    def experts_forward(self, y, picks, weights):
        order, ends = self.route(picks)
        rows = y[order // self.topk]
        a = torch.empty((rows.shape[0], self.inter), dtype=self.dtype, device="cuda")
        R.grouped_forward(self.up, rows, self.w_up, ends, a)
        h = torch.nn.functional.silu(a)
        d = torch.empty_like(rows)
        R.grouped_forward(self.down, h, self.w_down, ends, d)
        by_pick = torch.empty_like(d)
        by_pick[order] = d
        b = (by_pick.view(-1, self.topk, self.dim).float() * weights[:, :, None]).sum(1).to(self.dtype)
        return b, (order, ends, rows, a, h)

    def forward(self, x, y, picks, weights):
        b, kept = self.experts_forward(y, picks, weights)
        x_out, y_out = torch.empty_like(x), torch.empty_like(y)
        R.join_forward(self.join, x, b, self.w_post, self.gate, self.w_pre, x_out, y_out)
        return x_out, y_out, (b, x_out, weights, kept)

    def backward(self, dy_out, dx_out, kept):
        """The gradients of x, y and the weights for those of y' and x'."""
        b, x_out, weights, (order, ends, rows, a, h) = kept
        grads = {k: torch.empty(self.dim, dtype=torch.float32, device="cuda") for k in ("w_post", "gate", "w_pre")}
        dx, db = torch.empty_like(x_out), torch.empty_like(b)
        R.join_backward(self.join, dy_out, dx_out, x_out, b, self.w_post, self.gate, self.w_pre, dx, db,
                        grads["w_post"], grads["gate"], grads["w_pre"], self.join_ws)
        dd = (db[:, None, :].float() * weights[:, :, None]).to(self.dtype).view(-1, self.dim)[order]
        dh = torch.empty_like(h)
        R.grouped_backward_x(self.down, dd, self.w_down, ends, dh)
        grads["w_down"] = torch.empty(self.w_down.shape, dtype=torch.float32, device="cuda")
        R.grouped_backward_w(self.down_dw, dd, h, ends, grads["w_down"])
        s = torch.sigmoid(a.float())
        da = (dh.float() * s * (1 + a.float() * (1 - s))).to(self.dtype)
        drows = torch.empty_like(rows)
        R.grouped_backward_x(self.up, da, self.w_up, ends, drows)
        grads["w_up"] = torch.empty(self.w_up.shape, dtype=torch.float32, device="cuda")
        R.grouped_backward_w(self.up_dw, da, rows, ends, grads["w_up"])
        by_pick = torch.empty_like(drows)
        by_pick[order] = drows
        dy = by_pick.view(-1, self.topk, self.dim).float().sum(1).to(self.dtype)
        return dx, dy, grads


class Decode:
    """The same block for single tokens of many requests, with a shared projection that each request adapts."""

    def __init__(self, block, adapters, rank, tokens, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dim, t = block.dim, block.dtype
        self.block = block
        self.w = torch.randn((dim, dim), generator=g, device="cuda").mul_(dim ** -0.5).to(t)
        self.a = torch.randn((adapters, rank, dim), generator=g, device="cuda").mul_(dim ** -0.5).to(t)
        self.b = torch.randn((adapters, dim, rank), generator=g, device="cuda").mul_(rank ** -0.5).to(t)
        self.factor = torch.rand(adapters, generator=g, device="cuda") + 0.5
        self.plan = R.Adapters(self.a, self.b, self.factor)
        self.ws = torch.empty(R.adapter_workspace_bytes(self.plan, tokens), dtype=torch.uint8, device="cuda")

    def step(self, x, y, picks, weights, request):
        """request: int32 [tokens], each token's adapter or -1. x is updated in place."""
        b, _ = self.block.experts_forward(y, picks, weights)
        shared = torch.empty_like(y)
        R.adapter_project(self.plan, y, self.w, request, shared, self.ws)
        b += shared
        y_out = torch.empty_like(y)
        R.join_forward(self.block.join, x, b, self.block.w_post, self.block.gate, self.block.w_pre, x, y_out)
        return y_out


def inputs(block, tokens, seed=0):
    """A stream, its norm, and every token's picks with their weights."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((tokens, block.dim), generator=g, device="cuda").to(
        torch.float32 if block.join.residual_type == R.MOE_TYPE_F32 else block.dtype)
    y = torch.empty((tokens, block.dim), dtype=block.dtype, device="cuda")
    R.join_forward(block.join, x, None, None, None, block.w_pre, None, y)   # no block yet: the norm of x alone
    logits = torch.randn((tokens, block.experts), generator=g, device="cuda")
    top = logits.topk(block.topk)
    return x, y, top.indices, top.values.softmax(-1)


def timed(f, n=20):
    for _ in range(3):
        f()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(n):
        f()
    torch.cuda.synchronize()
    return (time.perf_counter() - t) / n


def main():
    block = Block(dim=4096, inter=2048, experts=32, topk=6, tokens=2048, residual=torch.float32)
    x, y, picks, weights = inputs(block, 2048)
    gx, gy = torch.randn_like(x), torch.randn_like(y)

    def train():
        _, _, kept = block.forward(x, y, picks, weights)
        return block.backward(gy, gx, kept)

    print(f"training step, 2048 tokens, 32 experts of 2048 x 4096: {timed(train) * 1e3:.2f} ms")
    decode = Decode(block, adapters=24, rank=32, tokens=48)
    x, y, picks, weights = inputs(block, 48, seed=1)
    request = torch.arange(48, dtype=torch.int32, device="cuda") % 25 - 1
    print(f"decode step, 48 tokens, 24 adapters: {timed(lambda: decode.step(x, y, picks, weights, request)) * 1e6:.0f} us")


if __name__ == "__main__":
    main()
