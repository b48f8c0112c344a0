"""The gated feed-forward calls refuse bad arguments and tensors that do not fit before any launch (CPU)."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests.test_block_arguments import HOST, INT32, ROWS, SMALL, TYPE, z
from tests.test_block_arguments import refused as refused_tensor
from tests.test_block_refusals import EINVAL, EUNSUPPORTED, Fake, P, refused

BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
CALLS = {"forward": lambda g, v=P, off=P, out=P, st=None: R.gated_forward(g, v, P, P, off, out, P, P, st, stream=0),
         "hidden": lambda g, v=P, off=P, out=P, st=None: R.gated_backward_h(g, v, P, P, P, off, out, P, None, st, stream=0),
         "input": lambda g, v=P, off=P, out=P, st=None: R.gated_backward_x(g, v, P, P, P, off, out, st, stream=0)}
ALL = set(CALLS)


def gated(**over):
    g = R.Gated(4, 64, 32, R.MOE_TYPE_FP16, dx=R.MOE_TYPE_F32)
    for k, v in over.items():
        setattr(g, k, v)
    return g


MOST = R.MOE_GROUPED_MAX_STRIDE + 1
BAD = [({"n_groups": 0}, EINVAL, ALL), ({"n_groups": R.MOE_GROUPED_MAX_GROUPS + 1}, EUNSUPPORTED, ALL),
       ({"n": 0}, EINVAL, ALL), ({"k": 0}, EINVAL, ALL), ({"k": -5}, EINVAL, ALL), ({"type": 2}, EINVAL, ALL),
       ({"type": 9}, EINVAL, ALL), ({"dx_type": 0}, EINVAL, ALL), ({"act": 2}, EINVAL, ALL), ({"act": -1}, EINVAL, ALL),
       ({"limit": -1.0}, EINVAL, ALL), ({"limit": float("nan")}, EINVAL, ALL), ({"limit": float("inf")}, EINVAL, ALL),
       ({"x_stride": 31}, EINVAL, {"forward", "input"}), ({"h_stride": 63}, EINVAL, {"forward", "hidden"}),
       ({"gate_stride": 63}, EINVAL, ALL), ({"y_stride": 31}, EINVAL, {"hidden"}),
       ({"w_stride": 31}, EINVAL, {"forward", "input"}), ({"w_group_stride": 64 * 32 - 1}, EINVAL, {"forward", "input"}),
       ({"down_stride": 63}, EINVAL, {"hidden"}), ({"down_group_stride": 64 * 32 - 1}, EINVAL, {"hidden"}),
       ({"x_stride": MOST}, EUNSUPPORTED, {"forward", "input"}), ({"gate_stride": MOST}, EUNSUPPORTED, ALL),
       ({"y_stride": MOST}, EUNSUPPORTED, {"hidden"}), ({"h_stride": MOST}, EUNSUPPORTED, {"forward", "hidden"}),
       ({"w_stride": MOST, "w_group_stride": 1 << 40}, EUNSUPPORTED, {"forward", "input"}),
       ({"down_stride": MOST, "down_group_stride": 1 << 40}, EUNSUPPORTED, {"hidden"})]


@pytest.mark.parametrize("over,code,calls", BAD, ids=lambda v: str(v) if not isinstance(v, set) else "")
def test_description(over, code, calls):
    for name in calls:
        refused(code, lambda: CALLS[name](gated(**over)))


@pytest.mark.parametrize("name", sorted(ALL))
def test_arguments(name):
    call, g = CALLS[name], gated()
    for bad in (dict(v=Fake(4097)), dict(off=Fake(4098)), dict(off=None), dict(out=None), dict(out=Fake(4097)),
                dict(st=Fake(4098))):
        refused(EINVAL, lambda: call(g, **bad))
    for rows in ((1 << 31) - 1, R.MOE_GROUPED_MAX_ROWS + 1):
        refused(EUNSUPPORTED, lambda: call(g, v=Fake(rows=rows)))
    refused(EINVAL, lambda: call(g, v=None))
    with pytest.raises(R.MoeError):
        call(R.Grouped(4, 64, 32, R.MOE_TYPE_FP16))   # another call's description
    if name == "input":
        refused(EINVAL, lambda: call(g, out=Fake(4098)))   # f32 on an address of 2 bytes


def test_what_goes_together():
    g = gated()
    refused(EINVAL, lambda: R.gated_forward(g, P, P, P, P, P, P, None, stream=0))
    refused(EINVAL, lambda: R.gated_forward(g, P, P, P, P, P, None, P, stream=0))
    refused(EINVAL, lambda: R.gated_forward(g, P, P, None, P, P, stream=0))
    refused(EINVAL, lambda: R.gated_backward_h(g, P, P, P, None, P, P, P, stream=0))
    refused(EINVAL, lambda: R.gated_backward_h(g, P, P, P, P, P, P, None, stream=0))
    refused(EINVAL, lambda: R.gated_backward_x(g, P, None, P, P, P, P, stream=0))
    L = R.lib()
    assert L.moe_gated_forward(None, 4096, 4096, 4096, 4096, 4, 4096, None, None, None, None) == EINVAL


def test_activation_names():
    assert R.act_code("silu") == R.MOE_ACT_SILU and R.act_code("gelu") == R.MOE_ACT_GELU and R.act_code(1) == 1
    for bad in ("relu", None, 1.0):
        with pytest.raises(R.MoeError):
            R.act_code(bad)
    assert R.Gated(1, 8, 8, BF16).limit == 0 and R.Gated(1, 8, 8, BF16, limit=7.0).limit == 7


G, N, K, ROWS_ = 3, 16, 24, 6
FWD = {"x": (ROWS_, K), "w_gate": (G, N, K), "w_up": (G, N, K), "offsets": (G + 1,), "h": (ROWS_, N), "gate": (ROWS_, N),
       "up": (ROWS_, N)}
HID = {"dy": (ROWS_, K), "w_down": (G, K, N), "gate": (ROWS_, N), "up": (ROWS_, N), "offsets": (G + 1,),
       "dgate": (ROWS_, N), "dup": (ROWS_, N), "h": (ROWS_, N)}
INP = {"dgate": (ROWS_, N), "dup": (ROWS_, N), "w_gate": (G, N, K), "w_up": (G, N, K), "offsets": (G + 1,),
       "dx": (ROWS_, K)}
TENSOR_CALLS = [(R.gated_forward, FWD), (R.gated_backward_h, HID), (R.gated_backward_x, INP)]


@pytest.mark.parametrize("call,shapes", TENSOR_CALLS, ids=lambda v: getattr(v, "__name__", ""))
def test_tensors(call, shapes):
    plan = R.Gated(G, N, K, BF16)
    for what, shape in shapes.items():
        args = {key: Fake(4096, ROWS_) for key in shapes}

        def given(t):
            return lambda: call(plan, *{**args, what: t}.values(), stream=0)

        if what == "offsets":
            refused_tensor(given(z(G + 1, dtype=torch.int64)), INT32, what)
            refused_tensor(given(z(G, dtype=torch.int32)), SMALL, what)
            refused_tensor(given(z(G + 1, dtype=torch.int32)), HOST, what)
            continue
        refused_tensor(given(z(*shape)), HOST, what)
        refused_tensor(given(z(*shape, dtype=torch.int16)), HOST, what)
        refused_tensor(given(z(*shape, dtype=FP16)), TYPE, what)
        refused_tensor(given(z(*shape[:-1], shape[-1] - 1)), SMALL, what)
        refused_tensor(given(z(*shape[:-1], 2 * shape[-1])), ROWS, what)
        refused_tensor(given(z(*shape[:-1], 2 * shape[-1])[..., ::2]), ROWS, what)
