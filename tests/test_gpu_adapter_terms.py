"""The sorted tokens' low-rank values u = factor A x as 16-bit terms, far from order one.

Tolerances. As in the tests of moe_adapter_project: steps * 2^-23 of the sum of
the absolute terms for the f32 sums, and one rounding of the output. u enters
the products with B in f32 (up to 64 tokens here) or as fp16 terms of u times a
power of two that brings the row's largest value to [2^14, 2^15): two terms
leave 2^-22 of each value, and half of fp16's smallest step, 2^-25, which is at
most 2^-39 of the row's largest value. W is zero in these tests, so that nothing
hides the low-rank part."""
import pytest
import torch

from tests import test_gpu_adapter as adapter
from tests.block_helpers import BF16, F32, FP16, assert_within, half_step

pytestmark = pytest.mark.gpu


def want(s, out):
    m, n, k, r = s["m"], s["n"], s["k"], s["rank"]
    x, a, b = s["x"].double().cpu(), s["a"].double().cpu().reshape(-1, r, k), s["b"].double().cpu().reshape(-1, n, r)
    factor, index = s["factor"].double().cpu(), s["index"].cpu()
    v, mag, left = (torch.zeros((m, n), dtype=torch.float64) for _ in range(3))
    for i in range(s["adapters"]):
        rows = (index == i).nonzero()[:, 0]
        if not rows.numel():
            continue
        u, u_mag = factor[i] * (x[rows] @ a[i].t()), factor[i] * (x[rows].abs() @ a[i].abs().t())
        v[rows], mag[rows] = u @ b[i].t(), u_mag @ b[i].abs().t()
        piece = 0.0 if m <= 64 else 2.0 ** -22
        left[rows] = (piece * u.abs() + 2.0 ** -39 * u.abs().amax(1, keepdim=True)) @ b[i].abs().t()
    steps = k / 32 + k / 256 + 3 * r + 40
    return v, half_step(out) * v.abs() + steps * 2.0 ** -23 * mag + left + (2.0 ** -25 if out == FP16 else 0.0)


def make(m, rank, seed, factor=1.0, low=1.0, high=1.0, order="mixed"):
    """A of size `low`, B of size `high`, fp16."""
    s = adapter.make(m, 136, 264, rank, 3, FP16, seed=seed, order=order)
    s["w"].zero_()
    s["a"] *= low
    s["b"] *= high
    s["factor"] *= factor
    return s


@pytest.mark.parametrize("m", [40, 100, 700])
@pytest.mark.parametrize("factor", [2.0 ** -10, 2.0 ** -16, 2.0 ** -24, 2.0 ** -90])
def test_small_factors(m, factor):
    for rank, order in ((16, "mixed"), (70, "segments")):
        s = make(m, rank, seed=m, factor=factor, low=2.0 ** -8, high=2.0 ** 10, order=order)
        for out in (F32, FP16):
            v, tol = want(s, out)
            assert_within(adapter.run(s, out), v, tol, f"m {m} rank {rank} factor {factor} {out}")


@pytest.mark.parametrize("m", [40, 100, 700])
@pytest.mark.parametrize("low,high", [(2.0 ** -14, 2.0 ** 10), (2.0 ** -10, 2.0 ** 8), (2.0 ** 10, 2.0 ** -10)])
def test_sizes_of_a_and_b(m, low, high):
    s = make(m, 40, seed=m, low=low, high=high)
    v, tol = want(s, F32)
    assert_within(adapter.run(s, F32), v, tol, f"m {m} A {low} B {high}")


@pytest.mark.parametrize("m", [40, 100, 700])
def test_small_values_beside_large_ones(m):
    """Ranks whose values are 2^-20 of the others', against a B that is as much larger."""
    s = make(m, 40, seed=m)
    a, b = s["a"].view(3, 40, 264), s["b"].view(3, 136, 40)
    a[:, ::2] *= 2.0 ** -10
    a[:, 1::2] *= 2.0 ** 6
    b[:, :, ::2] *= 2.0 ** 8
    b[:, :, 1::2] *= 2.0 ** -8
    v, tol = want(s, F32)
    assert_within(adapter.run(s, F32), v, tol, f"m {m}")


@pytest.mark.parametrize("m", [40, 700])
def test_large_values_beside_an_infinite_one(m):
    """A row of A that is infinite, beside values of u past fp16's range that B meets with the other sign: the
    infinity decides alone."""
    s = make(m, 16, seed=m, low=2.0 ** 11)
    x, a, b = s["x"], s["a"].view(3, 16, 264), s["b"].view(3, 136, 16)
    x.abs_()
    a.abs_()
    a[:, 3] = float("inf")
    b.copy_(-b.abs() - 2.0 ** -6)
    b[:, :, 3] = 1.0
    mine = s["index"] >= 0
    assert float((x.double().cpu() @ a[0, 4].double().cpu()).min()) > 65504
    y = adapter.run(s, F32)
    assert (y[mine] == float("inf")).all() and not y[~mine].any()
