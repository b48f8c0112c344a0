"""The microscaled 4-bit calls refuse bad arguments and tensors that do not fit before any launch (CPU)."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests.test_block_arguments import HOST, INT32, ROWS, SMALL, TYPE, z
from tests.test_block_arguments import refused as refused_tensor
from tests.test_block_refusals import EINVAL, EUNSUPPORTED, Fake, P, refused

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
MOST = R.MOE_GROUPED_MAX_STRIDE + 1


def changed(plan, over):
    for k, v in over.items():
        setattr(plan, k, v)
    return plan


# ---- rows -----------------------------------------------------------------------------------------
def rows(**over):
    return changed(R.MxRows(70, BF16), over)


ROW_CALLS = {"quantise": lambda p, x=P, codes=P, scales=P: R.mx_quantise(p, x, codes, scales, stream=0),
             "dequantise": lambda p, x=P, codes=P, scales=P: R.mx_dequantise(p, codes, scales, x, stream=0)}
BOTH_ROWS = pytest.mark.parametrize("call", ROW_CALLS.values(), ids=ROW_CALLS)


@BOTH_ROWS
@pytest.mark.parametrize("over,code", [({"k": 0}, EINVAL), ({"k": -1}, EINVAL), ({"k": R.MOE_MX_MAX_K + 1}, EUNSUPPORTED),
                                       ({"type": 3}, EINVAL), ({"type": -1}, EINVAL), ({"scale": 2}, EINVAL),
                                       ({"scale": -1}, EINVAL), ({"x_stride": 69}, EINVAL), ({"code_stride": 34}, EINVAL),
                                       ({"scale_stride": 2}, EINVAL)], ids=str)
def test_rows_description(call, over, code):
    p = rows(**over)
    if over.get("k", 0) > 70:
        p.x_stride = p.code_stride = p.scale_stride = p.k
    refused(code, lambda: call(p))


@BOTH_ROWS
def test_rows_arguments(call):
    for bad in (dict(x=Fake(4097)), dict(x=None), dict(codes=None), dict(scales=None)):
        refused(EINVAL, lambda: call(rows(), **bad))
    with pytest.raises(R.MoeError):
        call(R.Mx(1, 8, 70, BF16))   # another call's description
    most = R.MOE_MX_MAX_K
    wide = R.MxRows(most, BF16)
    many = Fake(rows=1 << 15)
    refused(EUNSUPPORTED, lambda: call(wide, x=many, codes=many, scales=many))   # 2^32 blocks
    L = R.lib()
    assert L.moe_mx_quantise(None, 4096, 4, 4096, 4096, None) == EINVAL


def test_scale_names():
    assert R.MxRows(8, BF16).scale == R.MOE_MX_FLOOR and R.MxRows(8, BF16, scale="ceil").scale == R.MOE_MX_CEIL
    for bad in ("nearest", None):
        with pytest.raises(R.MoeError):
            R.MxRows(8, BF16, scale=bad)


# ---- products -------------------------------------------------------------------------------------
def mx(**over):
    return changed(R.Mx(4, 64, 70, R.MOE_TYPE_F32), over)


CALLS = {"plain": lambda m, v=P, w=P, s=P, off=P, out=P, st=None: R.mx_forward(m, v, s, w, s, off, out, st, stream=0),
         "gated": lambda m, v=P, w=P, s=P, off=P, out=P, st=None: R.mx_gated(m, v, s, w, s, w, s, off, out, st, stream=0)}
BOTH = pytest.mark.parametrize("call", CALLS.values(), ids=CALLS)


@BOTH
@pytest.mark.parametrize("over,code", [
    ({"n_groups": 0}, EINVAL), ({"n_groups": R.MOE_GROUPED_MAX_GROUPS + 1}, EUNSUPPORTED), ({"n": 0}, EINVAL), ({"k": 0}, EINVAL),
    ({"k": R.MOE_MX_MAX_K + 1}, EUNSUPPORTED), ({"out_type": 3}, EINVAL), ({"x_stride": 34}, EINVAL),
    ({"x_scale_stride": 2}, EINVAL), ({"y_stride": 63}, EINVAL), ({"w_stride": 34}, EINVAL), ({"w_scale_stride": 2}, EINVAL),
    ({"w_group_stride": 64 * 35 - 1}, EINVAL), ({"w_scale_group_stride": 64 * 3 - 1}, EINVAL), ({"x_stride": MOST}, EUNSUPPORTED),
    ({"x_scale_stride": MOST}, EUNSUPPORTED), ({"y_stride": MOST}, EUNSUPPORTED),
    ({"w_stride": MOST, "w_group_stride": 1 << 40}, EUNSUPPORTED),
    ({"w_scale_stride": MOST, "w_scale_group_stride": 1 << 40}, EUNSUPPORTED)], ids=str)
def test_description(call, over, code):
    refused(code, lambda: call(mx(**over)))


@pytest.mark.parametrize("over", [{"act": 2}, {"act": -1}, {"limit": -1.0}, {"limit": float("nan")}, {"limit": float("inf")}], ids=str)
def test_activation(over):
    refused(EINVAL, lambda: CALLS["gated"](mx(**over)))


@BOTH
def test_arguments(call):
    for bad in (dict(off=Fake(4098)), dict(off=None), dict(out=None), dict(out=Fake(4098)), dict(st=Fake(4098)), dict(w=None),
                dict(s=None), dict(v=None)):
        refused(EINVAL, lambda: call(mx(), **bad))
    refused(EUNSUPPORTED, lambda: call(mx(), v=Fake(rows=R.MOE_GROUPED_MAX_ROWS + 1)))
    with pytest.raises(R.MoeError):
        call(R.Grouped(4, 64, 70, R.MOE_TYPE_FP16))   # another call's description


# ---- tensors --------------------------------------------------------------------------------------
G, N, K, M = 3, 16, 70, 6
X, W = {"x": (M, 35), "x_scale": (M, 3)}, {"w": (G, N, 35), "w_scale": (G, N, 3)}
GATES = {"w_gate": (G, N, 35), "w_gate_scale": (G, N, 3), "w_up": (G, N, 35), "w_up_scale": (G, N, 3)}
TENSOR_CALLS = [(R.mx_quantise, lambda: R.MxRows(K, BF16), {"x": (M, K), "codes": (M, 35), "scales": (M, 3)}),
                (R.mx_dequantise, lambda: R.MxRows(K, BF16), {"codes": (M, 35), "scales": (M, 3), "x": (M, K)}),
                (R.mx_forward, lambda: R.Mx(G, N, K, BF16), {**X, **W, "offsets": (G + 1,), "y": (M, N)}),
                (R.mx_gated, lambda: R.Mx(G, N, K, BF16), {**X, **GATES, "offsets": (G + 1,), "h": (M, N)})]


@pytest.mark.parametrize("call,plan,shapes", TENSOR_CALLS, ids=lambda v: getattr(v, "__name__", ""))
def test_tensors(call, plan, shapes):
    for what, shape in shapes.items():
        args = {key: Fake(4096, M) for key in shapes}

        def given(t):
            return lambda: call(plan(), *{**args, what: t}.values(), stream=0)

        if what == "offsets":
            refused_tensor(given(z(G + 1, dtype=torch.int64)), INT32, what)
            refused_tensor(given(z(G, dtype=torch.int32)), SMALL, what)
            continue
        elements = what in ("y", "h") or (call in (R.mx_quantise, R.mx_dequantise) and what == "x")
        t = BF16 if elements else U8
        refused_tensor(given(z(*shape, dtype=t)), HOST, what)
        refused_tensor(given(z(*shape, dtype=F32)), TYPE if elements else "", what)
        if not elements:
            other = torch.float8_e8m0fnu if "scale" in what else torch.float4_e2m1fn_x2
            refused_tensor(given(z(*shape, dtype=t).view(other)), HOST, what)
            wrong = torch.float4_e2m1fn_x2 if "scale" in what else torch.float8_e8m0fnu
            refused_tensor(given(z(*shape, dtype=t).view(wrong)), "", what)
            refused_tensor(given(z(*shape, dtype=torch.int8)), "", what)
        refused_tensor(given(z(*shape[:-1], shape[-1] - 1, dtype=t)), SMALL, what)
        refused_tensor(given(z(*shape[:-1], 2 * shape[-1], dtype=t)), ROWS, what)
        refused_tensor(given(z(*shape[:-1], 2 * shape[-1], dtype=t)[..., ::2]), ROWS, what)
