"""The gated activation and its gradient in 64 bits, and how far the kernels' f32 forms of them may be off."""
import math

import torch


def inner(z, act):
    """The logistic function's argument and its slope."""
    if act == "silu":
        return z, torch.ones_like(z)
    c = 2 * math.sqrt(2 / math.pi)
    return c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z ** 2)


def activation(z, act):
    """act(z) and its derivative."""
    v, slope = inner(z, act)
    s = torch.sigmoid(v)
    return z * s, s + z * s * torch.sigmoid(-v) * slope


def limited(g, u, limit):
    return (g.clamp(max=limit), u.clamp(-limit, limit)) if limit else (g, u)


def hidden(g, u, act, limit):
    gc, uc = limited(g, u, limit)
    return activation(gc, act)[0] * uc


def gradients(g, u, dh, act, limit):
    """Of g and u, for h's gradient dh."""
    gc, uc = limited(g, u, limit)
    a, slope = activation(gc, act)
    dg, du = dh * uc * slope, dh * a
    if limit:
        dg, du = torch.where(g > limit, 0.0, dg), torch.where(u.abs() > limit, 0.0, du)
    return dg, du


# s takes an exponential, a sum, a reciprocal and a product of f32, each within
# two steps of 2^-23, and an argument v rounded a few times: s changes by at most
# v s (1 - s) 2^-21 <= 2^-22 for it. So s is off by less than 2^-19, act by
# less than |z| 2^-19; the derivative's two terms stay below 1.2, off by 2^-17.
ACT = 2.0 ** -19
SLOPE = 2.0 ** -17
STEEPEST = 1.2   # of act', silu 1.0999, gelu 1.129
