"""Microscaled 4-bit floats in 64 bits."""
import torch

STEPS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def quantised(x, rule):
    """(codes [rows, (k + 1) // 2], scales [rows, (k + 31) // 32]) of rows on the CPU: each block's scale from its largest
    magnitude, each element the nearest step by comparing with all of them."""
    rows, k = x.shape
    blocks = -(-k // 32)
    v = torch.zeros((rows, blocks * 32), dtype=torch.float64)
    v[:, :k] = x.double()
    v = v.view(rows, blocks, 32)
    bad = ~v.isfinite().all(-1)
    top = v.abs().amax(-1)
    part, power = torch.frexp(torch.where(bad | (top == 0), 1.0, top))   # part in [1/2, 1)
    e = power - 3 + ((part > 0.75).int() if rule == "ceil" else 0)
    e = torch.where(top == 0, -127, e).clamp(min=-127)
    a = torch.ldexp(v.abs(), -e[..., None])
    away = (a[..., None] - STEPS).abs()
    nearest = away.amin(-1, keepdim=True)
    tied = away == nearest   # one step, or two of which the even one counts
    index = torch.arange(8)
    code = torch.where(tied, index, -1).amax(-1)
    low = torch.where(tied, index, 8).amin(-1)
    code = torch.where((code != low) & (code % 2 == 1), low, code)
    code = torch.where(bad[..., None] | a.isnan(), 0, code + 8 * torch.signbit(v).int())
    code = torch.where(bad[..., None], 0, code).view(rows, -1)
    code[:, k:] = 0
    pairs = code[:, 0::2] + 16 * code[:, 1::2]
    return pairs[:, :(k + 1) // 2].to(torch.uint8), torch.where(bad, 255, e + 127).to(torch.uint8)


def values(codes, scales, k):
    """What they stand for, in 64 bits on their device; NaN for scale 255."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., :k].long()
    steps = STEPS.to(codes.device)
    v = steps[c & 7] * torch.where(c > 7, -1.0, 1.0).double()
    s = scales.double()
    return v * torch.where(s == 255, float("nan"), torch.exp2(s - 127)).repeat_interleave(32, -1)[..., :k]
