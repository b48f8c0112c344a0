"""Block joins in place: rows of two strides are refused (CPU)."""
import pytest

import routing_quant_expert_amd as R
from tests.test_block_refusals import EINVAL, Fake, P


def at(addr, rows):
    return Fake(addr, rows)


def code(call):
    with pytest.raises(R.MoeError) as ei:
        call()
    return ei.value.code, str(ei.value)


@pytest.mark.parametrize("rows", [2, 300])
@pytest.mark.parametrize("over", [{"x_out_stride": 72}, {"x_stride": 80}, {"y_stride": 66}, {"b_stride": 128}],
                         ids=lambda v: next(iter(v)))
def test_two_strides_in_place(rows, over):
    j = R.Join(64, R.MOE_TYPE_BF16, **over)
    x, b, other = at(4096, rows), at(1 << 20, rows), at(1 << 30, rows)
    stream = "x_out_stride" in over or "x_stride" in over
    call = (lambda: R.join_forward(j, x, b, P, P, P, x, other, stream=0)) if stream else (
        lambda: R.join_forward(j, x, b, P, P, P, other, b, stream=0))
    got = code(call)
    assert got[0] == EINVAL and "two row strides" in got[1]
    if stream:
        got = code(lambda: R.join_backward(j, P, x, other, None, None, None, P, x, None, None, None, None, None, stream=0))
        assert got[0] == EINVAL and "two row strides" in got[1]
