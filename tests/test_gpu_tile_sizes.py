"""The gated and the 4-bit products at sizes that go through each of the smaller tiles, aligned and not (the largest have
tests of their own). Checks and tolerances are those of the operators' own tests."""
import pytest

from tests import test_gpu_gated as gated
from tests import test_gpu_mx as mx
from tests.block_helpers import BF16, F32, FP16

pytestmark = pytest.mark.gpu

# rows by group: hardly any, few, many
GROUPS = {"128x16": [0, 1, 2, 5] * 75, "128x64": [30, 1, 64, 0, 17, 65, 32, 31] * 5, "128x128": [500, 129, 0, 900, 640, 831]}
# n and k: outputs enough to fill the chip with these tiles, sums short enough for no larger ones
WIDTHS = {"128x16": {way: (264, 272) for way in gated.WAYS}, "128x64": {way: (520, 528) for way in gated.WAYS},
          "128x128": {"forward": (776, 264), "hidden": (1288, 264), "input": (264, 1288)}}
TILES = pytest.mark.parametrize("tile", GROUPS)


@TILES
@pytest.mark.parametrize("way", gated.WAYS)
@pytest.mark.parametrize("odd", [0, 1], ids=["aligned", "unaligned"])
def test_gated(tile, way, odd):
    n, k = WIDTHS[tile][way]
    t = (BF16, FP16)[odd]
    gated.CHECKS[way](gated.make(GROUPS[tile], n + odd, k + 2 * odd, t, seed=31, before=70, after=33, act=("silu", "gelu")[odd],
                                 dx=(t, F32)[odd]))


@TILES
@pytest.mark.parametrize("of_two", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("k", [640, 1408, 1051], ids=["short", "aligned", "unaligned"])
def test_mx(tile, of_two, k):
    n = {"128x16": 520, "128x64": 520, "128x128": 1288}[tile]
    pad = 0 if k % 32 else 16
    mx.check(mx.make(GROUPS[tile], n + k % 2, k, seed=32, pad=pad, offset=pad, before=70, after=33, out=(BF16, F32)[k % 2],
                     act=("silu", "gelu")[k % 2], limit=1.0), of_two)


@pytest.mark.parametrize("way", gated.WAYS)
def test_one_row(way):
    """A single token of one expert, and of a few."""
    for sizes in ([1], [1, 0, 1, 1], [0, 1, 0]):
        gated.CHECKS[way](gated.make(sizes, 520, 1056, BF16, seed=33))
