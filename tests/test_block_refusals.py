"""The operators beside the layer refuse bad arguments before any launch (CPU)."""
import ctypes

import pytest

import routing_quant_expert_amd as R

EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3


class Fake:
    """Stands in for a device tensor in calls that must fail validation."""

    def __init__(self, addr=4096, rows=4, n=1 << 40):
        self.addr, self.shape, self.n = addr, (rows, 64), n

    def data_ptr(self):
        return self.addr

    def numel(self):
        return self.n

    def element_size(self):
        return 1


P = Fake()


def refused(code, call):
    with pytest.raises(R.MoeError) as ei:
        call()
    assert ei.value.code == code, str(ei.value)


def join(**over):
    j = R.Join(64, R.MOE_TYPE_BF16, residual=R.MOE_TYPE_F32)
    for k, v in over.items():
        setattr(j, k, v)
    return j


JOIN_BAD = [({"dim": 0}, EINVAL), ({"dim": -3}, EINVAL), ({"dim": R.MOE_JOIN_MAX_DIM + 1}, EUNSUPPORTED),
            ({"type": 2}, EINVAL), ({"type": 7}, EINVAL), ({"residual_type": 1}, EINVAL), ({"gate_rows": 2}, EINVAL),
            ({"scale": float("inf")}, EINVAL), ({"scale": float("nan")}, EINVAL), ({"eps": 0.0}, EINVAL),
            ({"eps": -1e-6}, EINVAL), ({"eps": float("nan")}, EINVAL), ({"x_stride": 63}, EINVAL),
            ({"x_out_stride": 63}, EINVAL), ({"b_stride": 63}, EINVAL), ({"y_stride": 63}, EINVAL),
            ({"gate_rows": 1, "gate_stride": 63}, EINVAL)]


@pytest.mark.parametrize("over,code", JOIN_BAD, ids=lambda v: str(v))
def test_join_description(over, code):
    j = join(**over)
    if over.get("dim", 64) > 64:
        for k in ("x_stride", "x_out_stride", "b_stride", "y_stride", "gate_stride"):
            setattr(j, k, j.dim)
    refused(code, lambda: R.join_forward(j, P, P, P, P, P, P, P, stream=0))
    refused(code, lambda: R.join_backward(j, P, P, P, P, P, P, P, P, P, P, P, P, P, stream=0))
    assert R.join_workspace_bytes(j, 4) == 0


def test_join_arguments():
    j = join()
    odd, odd2 = Fake(4097), Fake(4098)
    f = R.join_forward
    for m, code in ((0, EINVAL), (1 << 22, EUNSUPPORTED)):
        refused(code, lambda: f(j, Fake(rows=m), P, P, P, P, P, P, stream=0))
        refused(code, lambda: R.join_backward(j, P, P, P, P, P, P, P, Fake(rows=m), P, P, P, P, P, stream=0))
        assert R.join_workspace_bytes(j, m) == 0
    assert R.join_workspace_bytes(j, (1 << 22) - 1) > 0
    calls = [lambda: f(j, P, P, P, P, P, None, P, stream=0),        # a block and nowhere to write the stream
             lambda: f(j, P, None, P, None, P, P, P, stream=0),     # a norm after no block
             lambda: f(j, P, None, None, P, P, P, P, stream=0),     # a gate on no block
             lambda: f(j, P, P, P, P, P, P, None, stream=0),        # w_pre without y
             lambda: f(j, P, P, P, P, None, P, P, stream=0),        # y without w_pre
             lambda: f(j, P, None, None, None, None, None, None, stream=0),
             lambda: f(j, odd2, P, P, P, P, P, P, stream=0),        # an f32 stream on an address of 2 bytes
             lambda: f(j, P, odd, P, P, P, P, P, stream=0),
             lambda: f(j, P, P, P, P, P, P, odd, stream=0)]
    b = R.join_backward
    calls += [lambda: b(j, None, None, P, P, P, P, P, P, P, P, P, P, P, stream=0),   # no gradient comes in
              lambda: b(j, P, P, None, P, P, P, P, P, P, P, P, P, P, stream=0),      # dy without the stream
              lambda: b(j, P, P, P, P, P, P, None, P, P, P, P, P, P, stream=0),      # dy without w_pre
              lambda: b(j, None, P, P, P, P, P, P, P, P, P, P, P, P, stream=0),      # dw_pre without dy
              lambda: b(j, P, P, P, P, None, P, P, P, P, P, P, P, P, stream=0),      # dw_post without w_post
              lambda: b(j, P, P, P, P, P, None, P, P, P, P, P, P, P, stream=0),      # dgate without a gate
              lambda: b(j, P, P, P, None, None, None, P, P, P, None, None, P, P, stream=0),   # db without a block
              lambda: b(j, P, P, P, P, P, P, P, P, P, P, P, P, None, stream=0),      # sums without a workspace
              lambda: b(j, P, P, P, P, P, P, P, P, P, P, P, P, Fake(4096 + 128), stream=0),
              lambda: b(j, P, P, P, P, P, P, P, P, odd, P, P, P, P, stream=0),
              lambda: b(j, P, P, P, P, P, P, P, P, P, odd2, P, P, P, stream=0)]
    for i, call in enumerate(calls):
        with pytest.raises(R.MoeError) as ei:
            call()
        assert ei.value.code == EINVAL, i
    small = Fake(n=R.join_workspace_bytes(j, 4) - 1)
    refused(EWORKSPACE, lambda: b(j, P, P, P, P, P, P, P, P, P, P, P, P, small, stream=0))
    L = R.lib()
    assert L.moe_join_forward(None, 4096, 4096, None, None, None, 1, 4096, None, None) == EINVAL
    assert L.moe_join_forward(ctypes.byref(j), None, 4096, None, None, None, 1, 4096, None, None) == EINVAL
    assert L.moe_join_backward(ctypes.byref(j), 4096, None, 4096, None, None, None, 4096, 1, None, None, None, None,
                               None, None, 0, None) == EINVAL


def test_type_codes():
    import torch
    assert [R.type_code(t) for t in (torch.bfloat16, torch.float16, torch.float32)] == [0, 1, 2]
    with pytest.raises(R.MoeError):
        R.type_code(torch.float64)


def grouped(**over):
    g = R.Grouped(4, 64, 32, R.MOE_TYPE_FP16, out=R.MOE_TYPE_F32)
    for k, v in over.items():
        setattr(g, k, v)
    return g


GROUPED_CALLS = [R.grouped_forward, R.grouped_backward_x, R.grouped_backward_w]
GROUPED_BAD = [({"n_groups": 0}, EINVAL), ({"n_groups": R.MOE_GROUPED_MAX_GROUPS + 1}, EUNSUPPORTED), ({"n": 0}, EINVAL),
               ({"k": -1}, EINVAL), ({"type": 2}, EINVAL), ({"out_type": 0}, EINVAL), ({"out_type": 3}, EINVAL),
               ({"x_stride": 31}, EINVAL), ({"y_stride": 63}, EINVAL), ({"w_stride": 31}, EINVAL),
               ({"w_group_stride": 63 * 32 + 31}, EINVAL), ({"x_stride": R.MOE_GROUPED_MAX_STRIDE + 1}, EUNSUPPORTED),
               ({"y_stride": R.MOE_GROUPED_MAX_STRIDE + 1}, EUNSUPPORTED),
               ({"w_stride": R.MOE_GROUPED_MAX_STRIDE + 1, "w_group_stride": 1 << 40}, EUNSUPPORTED)]


@pytest.mark.parametrize("over,code", GROUPED_BAD, ids=lambda v: str(v))
def test_grouped_description(over, code):
    for f in GROUPED_CALLS:
        refused(code, lambda: f(grouped(**over), P, P, P, P, stream=0))


def test_grouped_arguments():
    g = grouped()
    odd, odd2 = Fake(4097), Fake(4098)
    for f in GROUPED_CALLS:
        for i, a in enumerate(([None] * 4, [odd, P, P, P], [P, odd, P, P], [P, P, odd2, P], [P, P, None, P],
                               [P, P, P, None], [P, P, P, odd2], [P, None, P, P])):
            if a[0] is None:
                a[0] = Fake(0)
            refused(EINVAL, lambda: f(g, *a, stream=0))
        refused(EINVAL, lambda: f(g, P, P, P, P, status=odd2, stream=0))
        refused(EUNSUPPORTED, lambda: f(g, Fake(rows=1 << 31), P, P, P, stream=0))
        # more tiles than a launch can have
        if f is not R.grouped_backward_w:
            refused(EUNSUPPORTED, lambda: f(grouped(n=1 << 20, k=1 << 20, x_stride=1 << 20, y_stride=1 << 20, w_stride=1 << 20,
                                                    w_group_stride=1 << 40), Fake(rows=(1 << 31) - 1), P, P, P, stream=0))
    L = R.lib()
    assert L.moe_grouped_forward(None, 4096, 4096, 4096, 1, 4096, None, None) == EINVAL
    assert L.moe_grouped_forward(ctypes.byref(g), 4096, 4096, 4096, -1, 4096, None, None) == EINVAL
    # nothing to write: no pointers needed
    assert L.moe_grouped_forward(ctypes.byref(g), None, None, 4096, 0, None, None, None) == 0
    assert L.moe_grouped_forward(ctypes.byref(g), None, None, None, 0, None, None, None) == EINVAL


def adapters(**over):
    import torch
    p = R.Adapters(torch.zeros(3, 8, 32, dtype=torch.bfloat16), torch.zeros(3, 64, 8, dtype=torch.bfloat16), out=torch.float32)
    for k, v in over.items():
        setattr(p, k, v)
    return p


BIG = R.MOE_GROUPED_MAX_STRIDE + 1
ADAPTER_BAD = [({"n_adapters": 0}, EINVAL), ({"rank": 0}, EINVAL), ({"n": 0}, EINVAL), ({"k": 0}, EINVAL),
               ({"n_adapters": R.MOE_ADAPTER_MAX_ADAPTERS + 1}, EUNSUPPORTED),
               ({"rank": R.MOE_ADAPTER_MAX_RANK + 1}, EUNSUPPORTED), ({"type": 2}, EINVAL), ({"out_type": 1}, EINVAL),
               ({"x_stride": 31}, EINVAL), ({"w_stride": 31}, EINVAL), ({"a_stride": 31}, EINVAL),
               ({"b_stride": 7}, EINVAL), ({"out_stride": 63}, EINVAL), ({"a_group_stride": 8 * 32 - 1}, EINVAL),
               ({"b_group_stride": 64 * 8 - 1}, EINVAL), ({"a": None}, EINVAL), ({"b": None}, EINVAL),
               ({"a": 4097}, EINVAL), ({"b": 4097}, EINVAL), ({"factor": 4098}, EINVAL)]
ADAPTER_BAD += [({k: BIG, "a_group_stride": 1 << 40, "b_group_stride": 1 << 40}, EUNSUPPORTED)
                for k in ("x_stride", "w_stride", "out_stride", "a_stride", "b_stride")]


@pytest.mark.parametrize("over,code", ADAPTER_BAD, ids=lambda v: str(v))
def test_adapter_description(over, code):
    p = adapters(**over)
    refused(code, lambda: R.adapter_project(p, P, P, P, P, P, stream=0))
    assert R.adapter_workspace_bytes(p, 4) == 0


def test_adapter_arguments():
    import torch
    p = adapters()
    odd, odd2 = Fake(4097), Fake(4098)
    f = R.adapter_project
    for a in ([Fake(0), P, P, P], [P, None, P, P], [P, P, None, P], [P, P, P, None], [odd, P, P, P], [P, odd, P, P],
              [P, P, odd2, P], [P, P, P, odd2]):
        refused(EINVAL, lambda: f(p, *a, P, stream=0))
    refused(EINVAL, lambda: f(p, P, P, P, P, P, status=odd2, stream=0))
    refused(EINVAL, lambda: f(p, P, P, P, P, None, stream=0))
    refused(EINVAL, lambda: f(p, P, P, P, P, Fake(4096 + 128), stream=0))
    for m in (1, 64, 65, 1000, R.MOE_ADAPTER_MAX_TOKENS):
        need = R.adapter_workspace_bytes(p, m)
        assert need > 0 and need % 256 == 0
        if m != 64:
            continue
        refused(EWORKSPACE, lambda: f(p, Fake(rows=m), P, P, P, Fake(n=need - 1), stream=0))
    sizes = [R.adapter_workspace_bytes(p, m) for m in (1, 10, 64, 65, 200, 5000)]
    assert sizes == sorted(sizes)
    refused(EINVAL, lambda: f(p, Fake(rows=0), P, P, P, P, stream=0))
    refused(EUNSUPPORTED, lambda: f(p, Fake(rows=R.MOE_ADAPTER_MAX_TOKENS + 1), P, P, P, P, stream=0))
    L = R.lib()
    assert L.moe_adapter_project(None, 4096, 4096, 4096, 1, 4096, 4096, 1 << 30, None, None) == EINVAL
    a, b = torch.zeros(3, 8, 32, dtype=torch.bfloat16), torch.zeros(3, 64, 8, dtype=torch.bfloat16)
    for call in (lambda: R.Adapters(a, b[:2]), lambda: R.Adapters(a, b.half()), lambda: R.Adapters(a, b[:, :, :7]),
                 lambda: R.Adapters(a.transpose(1, 2).contiguous().transpose(1, 2), b),
                 lambda: R.Adapters(a, b, torch.zeros(3, dtype=torch.float16)),
                 lambda: R.Adapters(a, b, torch.zeros(4)), lambda: R.Adapters(a, b, torch.zeros(6)[::2]),
                 lambda: R.Adapters(a.double(), b.double())):
        refused(EINVAL, call)
