"""The grouped products and the adapter projection at sizes that take the larger
tiles, the streams of tiles and the sort of more than 4096 tokens. Values and
tolerances are those of the tests of each operator."""
import pytest
import torch

from tests import test_gpu_adapter as adapter
from tests import test_gpu_grouped as grouped
from tests.block_helpers import BF16, F32, FP16, padding_kept, strided

pytestmark = pytest.mark.gpu

RAGGED = [700, 0, 1, 901, 127, 128, 129, 640, 1100, 64, 900, 870]


def within(got, want, tol, what):
    """As assert_within, on the device."""
    assert torch.isfinite(got).all(), what
    assert float(((got.double() - want).abs() - tol).max()) <= 0, what


def check_grouped(s, way, out):
    y, store = grouped.output(s, way, out)
    grouped.call(s, way, y)
    torch.cuda.synchronize()
    assert padding_kept(y, store)
    v, mag, most = grouped.want(s, way)
    within(y, v, grouped.tolerance(v, mag, most, out), f"{way} {s['n']}x{s['k']}")


@pytest.mark.parametrize("way", ["forward", "dx"])
@pytest.mark.parametrize("wide,red", [(1544, 200), (1543, 201), (4096, 1032), (4104, 1096)])
def test_large_row_tiles(way, wide, red):
    n, k = (wide, red) if way == "forward" else (red, wide)
    odd = wide % 8 != 0
    s = grouped.make(RAGGED, n, k, BF16, seed=1, before=3, after=5, pad=1 if odd else 8, offset=1 if odd else 8)
    check_grouped(s, way, BF16)
    check_grouped(grouped.make(RAGGED, n, k, FP16, seed=2), way, F32)


@pytest.mark.parametrize("n,k", [(520, 1032), (512, 1024), (136, 3016), (1032, 264)])
def test_streams_of_weight_gradient_tiles(n, k):
    """Groups of no row, of less than a step, of whole steps, of a step and one row more, one after another."""
    sizes = ([0, 1, 63, 64, 65, 129, 200, 0, 0, 128, 192, 256, 31, 320, 5, 700] * 5)[:70]
    check_grouped(grouped.make(sizes, n, k, BF16, seed=3, before=2, after=1), "dw", BF16)
    check_grouped(grouped.make(sizes, n, k, FP16, seed=4, pad=8, offset=8), "dw", F32)


@pytest.mark.parametrize("sizes", [[5000], [0] * 200 + [70], [64] * 200, [1, 0] * 300], ids=lambda v: f"{len(v)}x{sum(v)}")
def test_streams_of_few_or_empty_groups(sizes):
    check_grouped(grouped.make(sizes, 264, 392, BF16, seed=5), "dw", F32)


def test_infinities_stay_in_their_group_in_a_stream():
    """A group's last step is filled up with rows that are not its own: none of the next group's values get in."""
    s = grouped.make([70, 65, 1, 130, 64] * 14, 520, 1032, BF16, seed=6)
    clean, _ = grouped.output(s, "dw", BF16)
    grouped.call(s, "dw", clean)
    n, g = 520, 6
    a, b = s["ends"][g], s["ends"][g + 1]
    s["x"][a:b], s["dy"][a:b] = float("nan"), float("inf")
    y, _ = grouped.output(s, "dw", BF16)
    grouped.call(s, "dw", y)
    assert y[g * n:(g + 1) * n].isnan().all()
    y[g * n:(g + 1) * n] = clean[g * n:(g + 1) * n]
    assert torch.equal(y, clean)


def check_adapter(s, out):
    y = adapter.run(s, out)
    v, tol = adapter.want(s, out)
    within(y, v, tol, f"m {s['m']} n {s['n']} k {s['k']}")
    return y


@pytest.mark.parametrize("m,n,k,rank,adapters", [(5000, 1032, 264, 24, 6), (5000, 1031, 263, 70, 5), (4096, 1024, 128, 8, 300),
                                                 (4097, 1024, 128, 8, 2), (8200, 2824, 1032, 16, 4)])
def test_many_tokens(m, n, k, rank, adapters):
    odd = n % 8 != 0
    check_adapter(adapter.make(m, n, k, rank, adapters, BF16, seed=m, pad=1 if odd else 8, offset=1 if odd else 8), F32)
    check_adapter(adapter.make(m, n, k, rank, adapters, FP16, seed=m, order="segments"), FP16)


def test_many_tokens_do_not_depend_on_their_places():
    s = adapter.make(5000, 1032, 264, 24, 6, BF16, seed=4)
    y = adapter.run(s, F32)
    assert torch.equal(y, adapter.run(s, F32))
    perm = torch.randperm(5000, generator=torch.Generator().manual_seed(1)).cuda()
    moved = {**s, "index": s["index"][perm].contiguous()}
    moved["x"] = strided(5000, 264, BF16)[0].copy_(s["x"][perm])
    assert torch.equal(adapter.run(moved, F32), y[perm])


@pytest.mark.parametrize("m", [100, 500])
def test_tokens_in_several_tiles_of_the_sliced_sums(m):
    for adapters in (1, 40):
        check_adapter(adapter.make(m, 264, 1544, 24, adapters, BF16, seed=m), F32)
        check_adapter(adapter.make(m, 263, 515, 9, adapters, FP16, seed=m, pad=1, offset=3), FP16)
