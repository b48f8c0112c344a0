"""The operators beside the layer refuse tensors that do not fit their description (CPU). Where a tensor lies is looked
at last, so a host tensor that fits is refused for that alone: it stands for the device tensor that would be taken."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests.test_block_refusals import EINVAL, Fake

BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
HOST = "not on the device"
TYPE = "not of the described element type"
SMALL = "smaller than"
ROWS = "its rows do not lie"
INT32 = "must be int32"


def refused(call, text, what=None):
    with pytest.raises(R.MoeError) as ei:
        call()
    assert ei.value.code == EINVAL, str(ei.value)
    assert text in str(ei.value), str(ei.value)
    if what:
        assert f" {what}:" in str(ei.value), str(ei.value)


def named(v):
    return v.replace(" ", "-") if isinstance(v, str) else str(v.dtype).split(".")[1] + "x".join(map(str, v.shape))


def z(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def base():
    """Memory that goes on behind what is cut from it."""
    return torch.zeros(1 << 16, dtype=BF16)


M, DIM = 4, 64
JOIN = ("x", "block", "w_post", "gate", "w_pre", "x_out", "y")


def join_forward(args, **plan):
    R.join_forward(R.Join(DIM, BF16, residual=F32, **plan), *(args[k] for k in JOIN), stream=0)


JOIN_BAD = [("x", z(M, DIM), TYPE), ("x", z(M, DIM, dtype=torch.float64), TYPE), ("block", z(M, DIM, dtype=FP16), TYPE),
            ("block", z(M - 1, DIM), SMALL), ("block", base()[:3 * DIM].view(3, DIM), ROWS), ("y", z(M, DIM - 1), SMALL),
            ("y", z(M, 2 * DIM), ROWS), ("y", z(M, 2 * DIM)[:, ::2], ROWS), ("y", z(DIM, M).t(), ROWS),
            ("x", z(1, DIM, dtype=F32).expand(M, DIM), SMALL), ("block", base()[:DIM].view(1, DIM).expand(M, DIM), ROWS),
            ("w_post", z(DIM - 1), SMALL), ("w_post", base()[:DIM - 1], ROWS), ("gate", z(2 * DIM)[::2], ROWS),
            ("w_pre", z(DIM, dtype=FP16), TYPE), ("x_out", z(M, DIM // 2, dtype=F32), SMALL),
            ("x_out", z(M, DIM, dtype=torch.complex64), TYPE)]


@pytest.mark.parametrize("i", range(len(JOIN_BAD)))
def test_join_forward(i):
    what, bad, text = JOIN_BAD[i]
    refused(lambda: join_forward({**{k: Fake(4096, M) for k in JOIN}, what: bad}), text, what)


# flat memory, the bits as integers, rows of a wider table, more rows than needed, another split of the same rows, one row
JOIN_GOOD = [("x", z(M, DIM, dtype=F32)), ("block", z(M, DIM, dtype=torch.int16)), ("block", z(M, 2 * DIM, dtype=torch.uint8)),
             ("y", z(M * DIM)), ("y", z(M + 3, DIM)), ("block", z(M, 4, DIM // 4)), ("y", z(2, 2, DIM)), ("gate", z(1, DIM)),
             ("w_pre", z(DIM + 5)), ("w_post", base()[3:3 + DIM])]


@pytest.mark.parametrize("i", range(len(JOIN_GOOD)))
def test_join_forward_takes(i):
    what, good = JOIN_GOOD[i]
    refused(lambda: join_forward({**{k: Fake(4096, M) for k in JOIN}, what: good}), HOST, what)


def test_join_strides():
    wide = z(M, 100)
    args = {k: Fake(4096, M) for k in JOIN}
    refused(lambda: join_forward({**args, "block": wide[:, :DIM]}, b_stride=100), HOST, "block")
    refused(lambda: join_forward({**args, "block": wide[:, 36:]}, b_stride=100), HOST, "block")
    refused(lambda: join_forward({**args, "block": wide[:, :DIM]}), ROWS, "block")
    refused(lambda: join_forward({**args, "block": wide[:, 37:]}, b_stride=100), SMALL, "block")
    refused(lambda: join_forward({**args, "gate": z(DIM)}, gate_rows=True), SMALL, "gate")
    refused(lambda: join_forward({**args, "gate": z(M, DIM)}, gate_rows=True), HOST, "gate")
    one = {k: Fake(4096, 1) for k in JOIN}
    refused(lambda: join_forward({**one, "block": wide[1:2, :DIM]}), HOST, "block")       # one row: its stride says nothing
    refused(lambda: join_forward({**one, "block": wide[1:2, :DIM - 1]}), ROWS, "block")
    refused(lambda: join_forward({**one, "x": torch.zeros((), dtype=F32)}), "has no rows", "x")
    refused(lambda: join_forward({**one, "x": None}), "must not be None", "x")
    refused(lambda: join_forward({**one, "x": z(DIM, dtype=F32)}), SMALL, "x")            # 64 rows of one element


BACK = ("dy", "dx_out", "x_out", "block", "w_post", "gate", "w_pre", "dx", "dblock", "dw_post", "dgate", "dw_pre", "ws")


@pytest.mark.parametrize("what,bad,text", [
    ("dy", z(M, DIM, dtype=F32), TYPE), ("dx_out", z(M, DIM), TYPE), ("x_out", z(M - 1, DIM, dtype=F32), SMALL),
    ("dx", z(M, DIM), TYPE), ("dblock", z(M, DIM + 8), ROWS), ("dw_post", z(DIM), TYPE), ("dw_pre", z(DIM - 1, dtype=F32), SMALL),
    ("dgate", z(DIM), TYPE), ("ws", z(1 << 16)[::2], "not contiguous"), ("ws", z(1 << 16), HOST),
    ("dgate", z(DIM, dtype=F32), HOST), ("dx", z(M, DIM, dtype=F32), HOST), ("dblock", z(M, DIM), HOST)], ids=named)
def test_join_backward(what, bad, text):
    args = {k: Fake(4096, M) for k in BACK}
    args[what] = bad
    refused(lambda: R.join_backward(R.Join(DIM, BF16, residual=F32), *(args[k] for k in BACK), stream=0), text,
            "workspace" if what == "ws" else what)


G, N, K, RN = 3, 40, 24, 10
WAYS = {"forward": (R.grouped_forward, ("x", "w", "offsets", "y")), "dx": (R.grouped_backward_x, ("dy", "w", "offsets", "dx")),
        "dw": (R.grouped_backward_w, ("dy", "x", "offsets", "dw"))}
SHAPES = {"x": (RN, K), "dx": (RN, K), "y": (RN, N), "dy": (RN, N), "w": (G, N, K), "dw": (G, N, K)}


def grouped(way, over, status=None, **plan):
    call, names = WAYS[way]
    args = {k: Fake(4096, RN) for k in names}
    args.update(over)
    call(R.Grouped(G, N, K, BF16, **plan), *(args[k] for k in names), status=status, stream=0)


@pytest.mark.parametrize("way", WAYS)
def test_grouped(way):
    for off in (torch.zeros(G + 1, dtype=torch.int64), torch.zeros(G + 1, dtype=F32), torch.zeros(G + 1, dtype=torch.int16)):
        refused(lambda: grouped(way, {"offsets": off}), INT32, "offsets")
    refused(lambda: grouped(way, {"offsets": z(G, dtype=torch.int32)}), SMALL, "offsets")
    refused(lambda: grouped(way, {"offsets": z(9, dtype=torch.int32)[:G]}), ROWS, "offsets")
    refused(lambda: grouped(way, {"offsets": z(2 * G + 2, dtype=torch.int32)[::2]}), ROWS, "offsets")
    refused(lambda: grouped(way, {"offsets": z(G + 1, dtype=torch.int32)}), HOST, "offsets")
    refused(lambda: grouped(way, {}, status=z(1, dtype=torch.int64)), INT32, "status")
    refused(lambda: grouped(way, {}, status=z(1, dtype=torch.int32)), HOST, "status")
    for what in WAYS[way][1]:
        if what == "offsets":
            continue
        shape = SHAPES[what]
        good = [z(*shape), z(*shape, dtype=torch.uint16), z(shape[0] * 100, *shape[1:])[:shape[0]]]
        bad = [(z(*shape, dtype=FP16), TYPE), (z(*shape[:-1], shape[-1] + 1), ROWS), (z(*shape[:-1], 2 * shape[-1])[..., ::2], ROWS),
               (z(*shape[:-1], shape[-1] - 1), SMALL)]
        if what not in ("x", "dy") or (way == "dw" and what == "x"):   # (the first operand's rows are the call's)
            bad += [(z(shape[0] - 1, *shape[1:]), SMALL), (z(shape[0] * 100, *shape[1:])[:shape[0] - 1], ROWS)]
            good += [z(*shape).flatten(), z(shape[0] + 2, *shape[1:])]
        if what in ("w", "dw"):
            good += [z(G * N, K)]
            bad += [(z(G, K, N).transpose(1, 2), ROWS), (z(1, N, K).expand(G, N, K), SMALL)]
        for t in good:
            refused(lambda: grouped(way, {what: t}), HOST, what)
        for t, text in bad:
            refused(lambda: grouped(way, {what: t}), text, what)


def test_grouped_strides():
    w = z(G, N + 2, K + 8)
    stride = {"w_stride": K + 8, "w_group_stride": (N + 2) * (K + 8)}
    refused(lambda: grouped("forward", {"w": w[:, :N, :K]}, **stride), HOST, "w")
    refused(lambda: grouped("forward", {"w": w[:, :N, :K]}, w_stride=K + 8), ROWS, "w")
    refused(lambda: grouped("forward", {"w": z(G * N, K + 8)[:, :K]}, w_stride=K + 8), HOST, "w")
    refused(lambda: grouped("forward", {"w": z(G * N, K + 8)[:, :K]}, w_stride=K + 8, w_group_stride=N * (K + 8) + 1), ROWS, "w")
    refused(lambda: grouped("forward", {"x": z(RN, K + 4)[:, :K]}, x_stride=K + 4), HOST, "x")
    refused(lambda: grouped("forward", {"y": z(RN + 5, N + 4)[:, :N]}, y_stride=N + 4), HOST, "y")
    refused(lambda: grouped("forward", {"y": z(RN, N, dtype=BF16)}, out=F32), TYPE, "y")


def adapter(over):
    args = {**{k: Fake(4096, M) for k in ("x", "w", "index", "out", "ws")}, **over}
    R.adapter_project(R.Adapters(z(2, 8, K), z(2, N, 8)), *args.values(), stream=0)


@pytest.mark.parametrize("what,bad,text", [
    ("index", z(M, dtype=torch.int64), INT32), ("index", z(M - 1, dtype=torch.int32), SMALL),
    ("index", z(M + 9, dtype=torch.int32)[:M - 1], ROWS), ("index", z(M, 2, dtype=torch.int32)[:, 0], ROWS),
    ("x", z(M, K, dtype=FP16), TYPE), ("x", z(M, K + 8), ROWS), ("x", z(K, M).t(), ROWS), ("w", z(N - 1, K), SMALL),
    ("w", z(K, N).t(), ROWS), ("out", z(M - 1, N), SMALL), ("out", z(M, N, dtype=F32), TYPE), ("out", z(M, 2 * N), ROWS),
    ("index", z(M, dtype=torch.int32), HOST), ("index", z(M, 1, dtype=torch.int32), HOST), ("x", z(M, K), HOST),
    ("w", z(N, K), HOST), ("out", z(M, N), HOST), ("ws", z(64), HOST)], ids=named)
def test_adapter(what, bad, text):
    refused(lambda: adapter({what: bad}), text, "workspace" if what == "ws" else what)


def test_another_calls_description():
    j, g = R.Join(DIM, BF16), R.Grouped(G, N, K, BF16)
    f = [Fake()] * 13
    refused(lambda: R.join_forward(g, *f[:7], stream=0), "not the description")
    refused(lambda: R.grouped_forward(j, *f[:4], stream=0), "not the description")
    refused(lambda: R.adapter_project(g, *f[:5], stream=0), "not the description")
