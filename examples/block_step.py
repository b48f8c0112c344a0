"""The operators beside the layer as a model runs them together: a training step
and a decode step of one block with experts on 16-bit weights, or on weights in microscaled 4-bit floats.

    y            the normed residual stream
    rows         y's rows, one per (token, pick), sorted by expert
    h, d         h = silu(W_up[e] row), d = W_down[e] h        grouped products
                 h = silu(W_gate[e] row) * (W_up[e] row)       gated products (and of 4-bit operands)
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
        d, kept = self.rows_forward(rows, ends)
        by_pick = torch.empty_like(d)
        by_pick[order] = d
        b = (by_pick.view(-1, self.topk, self.dim).float() * weights[:, :, None]).sum(1).to(self.dtype)
        return b, (order, ends, rows, *kept)

    def rows_forward(self, rows, ends):
        """d of the sorted rows, and what their gradients need."""
        a = torch.empty((rows.shape[0], self.inter), dtype=self.dtype, device="cuda")
        R.grouped_forward(self.up, rows, self.w_up, ends, a)
        h = torch.nn.functional.silu(a)
        d = torch.empty_like(rows)
        R.grouped_forward(self.down, h, self.w_down, ends, d)
        return d, (a, h)

    def forward(self, x, y, picks, weights):
        b, kept = self.experts_forward(y, picks, weights)
        x_out, y_out = torch.empty_like(x), torch.empty_like(y)
        R.join_forward(self.join, x, b, self.w_post, self.gate, self.w_pre, x_out, y_out)
        return x_out, y_out, (b, x_out, weights, kept)

    def backward(self, dy_out, dx_out, kept):
        """The gradients of x, y and the weights for those of y' and x'."""
        b, x_out, weights, (order, ends, rows, *kept) = kept
        grads = {k: torch.empty(self.dim, dtype=torch.float32, device="cuda") for k in ("w_post", "gate", "w_pre")}
        dx, db = torch.empty_like(x_out), torch.empty_like(b)
        R.join_backward(self.join, dy_out, dx_out, x_out, b, self.w_post, self.gate, self.w_pre, dx, db,
                        grads["w_post"], grads["gate"], grads["w_pre"], self.join_ws)
        dd = (db[:, None, :].float() * weights[:, :, None]).to(self.dtype).view(-1, self.dim)[order]
        drows = self.rows_backward(dd, rows, ends, kept, grads)
        by_pick = torch.empty_like(drows)
        by_pick[order] = drows
        dy = by_pick.view(-1, self.topk, self.dim).float().sum(1).to(self.dtype)
        return dx, dy, grads

    def rows_backward(self, dd, rows, ends, kept, grads):
        """The sorted rows' gradient for d's; the weights' go into grads."""
        a, h = kept
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
        return drows


class GatedBlock(Block):
    """The block with gated experts."""

    def __init__(self, dim, inter, experts, topk, tokens, dtype=torch.bfloat16, limit=7.0, seed=0, **other):
        super().__init__(dim, inter, experts, topk, tokens, dtype=dtype, seed=seed, **other)
        g = torch.Generator(device="cuda").manual_seed(seed + 100)
        self.w_gate = torch.randn(self.w_up.shape, generator=g, device="cuda").mul_(dim ** -0.5).to(dtype)
        self.gated = R.Gated(experts, inter, dim, dtype, limit=limit)

    def rows_forward(self, rows, ends):
        h, gate, up = (torch.empty((rows.shape[0], self.inter), dtype=self.dtype, device="cuda") for _ in range(3))
        R.gated_forward(self.gated, rows, self.w_gate, self.w_up, ends, h, gate, up)
        d = torch.empty_like(rows)
        R.grouped_forward(self.down, h, self.w_down, ends, d)
        return d, (gate, up)

    def rows_backward(self, dd, rows, ends, kept, grads):
        gate, up = kept
        h, drows = torch.empty_like(gate), torch.empty_like(rows)
        R.gated_backward_h(self.gated, dd, self.w_down, gate, up, ends, gate, up, h)   # their gradients in place
        R.gated_backward_x(self.gated, gate, up, self.w_gate, self.w_up, ends, drows)
        for key, plan, dy, x in (("w_down", self.down_dw, dd, h), ("w_gate", self.up_dw, gate, rows), ("w_up", self.up_dw, up, rows)):
            grads[key] = torch.empty(getattr(self, key).shape, dtype=torch.float32, device="cuda")
            R.grouped_backward_w(plan, dy, x, ends, grads[key])
        return drows


class FourBitBlock(GatedBlock):
    """The gated block for serving, its experts and the rows that they read in microscaled 4-bit floats."""

    def __init__(self, dim, inter, experts, topk, tokens, dtype=torch.bfloat16, limit=7.0, **other):
        super().__init__(dim, inter, experts, topk, tokens, dtype=dtype, limit=limit, **other)
        self.four_gate, self.four_up, self.four_down = (self.in_4_bits(w) for w in (self.w_gate, self.w_up, self.w_down))
        self.mx_gated = R.Mx(experts, inter, dim, dtype, limit=limit)
        self.mx_down = R.Mx(experts, dim, inter, dtype)

    @staticmethod
    def in_4_bits(v):
        k = v.shape[-1]
        codes = torch.empty((*v.shape[:-1], (k + 1) // 2), dtype=torch.uint8, device="cuda")
        scales = torch.empty((*v.shape[:-1], (k + 31) // 32), dtype=torch.uint8, device="cuda")
        R.mx_quantise(R.MxRows(k, v.dtype, scale="ceil"), *(m.flatten(0, -2) for m in (v, codes, scales)))
        return codes, scales

    def rows_forward(self, rows, ends):
        row = self.in_4_bits(rows)
        h = torch.empty((rows.shape[0], self.inter), dtype=self.dtype, device="cuda")
        R.mx_gated(self.mx_gated, *row, *self.four_gate, *self.four_up, ends, h)
        four = self.in_4_bits(h)
        d = torch.empty_like(rows)
        R.mx_forward(self.mx_down, *four, *self.four_down, ends, d)
        return d, (row, h, four)


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
    for kind, what in ((Block, "experts"), (GatedBlock, "gated experts"), (FourBitBlock, "gated experts in 4 bits")):
        block = kind(dim=4096, inter=2048, experts=32, topk=6, tokens=2048, residual=torch.float32)
        if kind is not FourBitBlock:
            x, y, picks, weights = inputs(block, 2048)
            gx, gy = torch.randn_like(x), torch.randn_like(y)

            def train():
                _, _, kept = block.forward(x, y, picks, weights)
                return block.backward(gy, gx, kept)

            print(f"training step, 2048 tokens, 32 {what} of 2048 x 4096: {timed(train) * 1e3:.2f} ms")
        decode = Decode(block, adapters=24, rank=32, tokens=48)
        x, y, picks, weights = inputs(block, 48, seed=1)
        request = torch.arange(48, dtype=torch.int32, device="cuda") % 25 - 1
        print(f"decode step, 48 tokens, 32 {what}, 24 adapters: "
              f"{timed(lambda: decode.step(x, y, picks, weights, request)) * 1e6:.0f} us")


if __name__ == "__main__":
    main()
