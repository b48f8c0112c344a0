"""Limits of the operators beside the layer that their kernels' 32-bit row numbers need (CPU)."""
import pytest

import routing_quant_expert_amd as R
from tests.test_block_refusals import EUNSUPPORTED, GROUPED_CALLS, Fake, P, grouped, refused


@pytest.mark.parametrize("rows", [(1 << 31) - 1, (1 << 31) - 64, (1 << 31) - 255])
@pytest.mark.parametrize("call", GROUPED_CALLS, ids=lambda f: f.__name__)
def test_rows_that_no_tile_can_round_up(call, rows):
    """A group of so many rows, rounded up to steps of 64 or tiles of 128, would pass 2^31 and count as empty."""
    refused(EUNSUPPORTED, lambda: call(grouped(), Fake(rows=rows), P, P, P, stream=0))


def test_the_limit_itself_can_be_rounded_up():
    assert R.MOE_GROUPED_MAX_ROWS + 255 < 1 << 31
