"""The gated feed-forward calls look at the strides of the tensors that they are given (CPU: no rows, so nothing is launched)."""
import pytest

import routing_quant_expert_amd as R
from tests.test_block_refusals import EINVAL, EUNSUPPORTED, Fake, P, refused
from tests.test_gated_refusals import MOST, gated

NONE = Fake(rows=0)


@pytest.mark.parametrize("stride,code", [(0, EINVAL), (63, EINVAL), (-1, EINVAL), (MOST, EUNSUPPORTED)])
def test_forward_without_gate_and_up(stride, code):
    """What a program that only serves leaves unset, or has for another call."""
    R.gated_forward(gated(gate_stride=stride), NONE, P, P, P, P, stream=0)
    for gate, up in ((P, P), (P, None), (None, P)):
        refused(code, lambda: R.gated_forward(gated(gate_stride=stride), NONE, P, P, P, P, gate, up, stream=0))


@pytest.mark.parametrize("over", [{"y_stride": 0}, {"down_stride": 0}, {"down_group_stride": 0}, {"y_stride": MOST}], ids=str)
def test_strides_of_the_other_way(over):
    R.gated_forward(gated(**over), NONE, P, P, P, P, P, P, stream=0)
    R.gated_backward_x(gated(**over), NONE, P, P, P, P, P, stream=0)


@pytest.mark.parametrize("over", [{"x_stride": 0}, {"w_stride": 0}, {"w_group_stride": 0}, {"x_stride": MOST}], ids=str)
def test_strides_of_the_forward_weights(over):
    R.gated_backward_h(gated(**over), NONE, P, P, P, P, P, P, stream=0)
