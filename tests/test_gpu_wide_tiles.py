"""The grouped products of the gated feed-forward and of 4-bit operands at the sizes that go through the largest tiles:
every partial tile, more groups than a wave has lanes, rows of no group, and values that must stay in their group. Checks
and tolerances are those of the operators' own tests."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests import test_gpu_gated as gated
from tests import test_gpu_mx as mx
from tests.block_helpers import BF16, F32, FP16, padding_kept

pytestmark = pytest.mark.gpu

# 70 groups; tiles of 256 rows end after 1 to 256 of them, and so do their quarters of 64
EDGES = [1, 17, 64, 65, 100, 129, 192, 193, 256, 257, 300, 512, 0, 31] * 5
WIDTHS = {"forward": (1288, 1024), "hidden": (2568, 1024), "input": (1024, 2568)}   # (n, k): the last tile of columns has 8
PLAIN_GATED = pytest.mark.parametrize("of_two", [False, True], ids=["plain", "gated"])


@pytest.mark.parametrize("way", gated.WAYS)
@pytest.mark.parametrize("t,act", [(BF16, "silu"), (FP16, "gelu")], ids=["bf16", "fp16"])
def test_edges(way, t, act):
    gated.CHECKS[way](gated.make(EDGES, *WIDTHS[way], t, seed=21, pad=8, offset=8, before=300, after=261, act=act, dx=F32))


@PLAIN_GATED
@pytest.mark.parametrize("out,act", [(BF16, "gelu"), (F32, "silu")], ids=["bf16", "f32"])
def test_edges_in_4_bits(of_two, out, act):
    mx.check(mx.make(EDGES, 1288 if of_two else 2568, 2048, seed=22, pad=16, offset=16, before=300, after=261, out=out, act=act,
                     limit=1.0), of_two)


@pytest.mark.parametrize("way", gated.WAYS)
@pytest.mark.parametrize("terms", [256, 320])
def test_short_sums(way, terms):
    """The shortest sums that these tiles take: the pipeline's start and end with hardly a step between them."""
    n, k = (terms, 2568) if way == "input" else (1288 if way == "forward" else 2568, terms)
    gated.CHECKS[way](gated.make(EDGES, n, k, BF16, seed=30, before=5, after=7))


@PLAIN_GATED
def test_one_group_of_scales_in_4_bits(of_two):
    mx.check(mx.make(EDGES, 1288 if of_two else 2568, 1024, seed=30, before=5, after=7), of_two)


@pytest.mark.parametrize("way", ["hidden", "input"])
def test_few_rows_of_many_groups(way):
    sizes = [0, 1, 2, 5] * 75
    gated.CHECKS[way](gated.make(sizes, *((264, 1024) if way == "hidden" else (1024, 264)), BF16, seed=23, before=3, after=9))


@pytest.mark.parametrize("way", gated.WAYS)
@pytest.mark.parametrize("sizes", [[30, 7, 55], [500, 270, 2700, 900]], ids=["small", "large"])
def test_values_stay_in_their_group(way, sizes):
    """Infinities and NaN in the rows and the weights of one group leave the other groups' outputs as they were."""
    n, k = WIDTHS[way] if len(sizes) > 3 else (72, 136)
    s = gated.make(sizes, n, k, BF16, seed=24)

    def run():
        h, gate, up = (torch.full((s["rows"], n), 3.0, dtype=BF16, device="cuda") for _ in range(3))
        dx = torch.full((s["rows"], k), 3.0, dtype=BF16, device="cuda")
        if way == "forward":
            R.gated_forward(s["plan"], s["x"], s["w_gate"], s["w_up"], s["off"], h, gate, up)
            return h, gate, up
        if way == "hidden":
            R.gated_backward_h(s["plan"], s["dy"], s["w_down"], s["gate"], s["up"], s["off"], gate, up, h)
            return h, gate, up
        R.gated_backward_x(s["plan"], s["dgate"], s["dup"], s["w_gate"], s["w_up"], s["off"], dx)
        return (dx,)

    want = run()
    a, b = s["ends"][1], s["ends"][2]
    for bad in (float("nan"), float("inf")):
        for key in ("x", "dy", "dgate", "dup", "gate", "up"):
            s[key][a:b] = bad
        for key in ("w_gate", "w_up"):
            s[key].view(len(sizes), n, k)[1] = bad
        s["w_down"].view(len(sizes), k, n)[1] = bad
        for got, kept in zip(run(), want):
            assert torch.equal(got[:a], kept[:a]) and torch.equal(got[b:], kept[b:])


@PLAIN_GATED
@pytest.mark.parametrize("sizes,n,k", [([30, 7, 55], 72, 160), ([500, 270, 2700, 900], 2568, 2048)], ids=["small", "large"])
def test_nan_stays_in_its_group_in_4_bits(of_two, sizes, n, k):
    s = mx.make(sizes, n, k, seed=25)
    want = mx.run(s, of_two)
    a, b = s["ends"][1], s["ends"][2]
    s["x"][1][a:b] = 255
    for _, scale in (s["w"], s["w2"]):
        scale.view(len(sizes), n, -1)[1] = 255
    got = mx.run(s, of_two)
    assert torch.equal(got[:a], want[:a]) and torch.equal(got[b:], want[b:]) and got[a:b].isnan().all()


@pytest.mark.parametrize("ends", [[0, 5000, 3000, 9000], [0, 4000, 6144, 8000], [-2, 4000, 6000, 6144], [6144, 3000, 1000, 0]])
def test_bad_offsets_are_reported(ends):
    sizes = [2048] * 3
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    for way, (n, k) in WIDTHS.items():
        s = gated.make(sizes, n, k, BF16, seed=26, pad=8)
        outs = [gated.output(s, n, BF16) for _ in range(3)]
        dx, st = gated.output(s, k, BF16), gated.status_word()
        if way == "forward":
            R.gated_forward(s["plan"], s["x"], s["w_gate"], s["w_up"], off, *(v for v, _ in outs), status=st)
        elif way == "hidden":
            R.gated_backward_h(s["plan"], s["dy"], s["w_down"], s["gate"], s["up"], off, *(v for v, _ in outs), status=st)
        else:
            R.gated_backward_x(s["plan"], s["dgate"], s["dup"], s["w_gate"], s["w_up"], off, dx[0], status=st)
        torch.cuda.synchronize()
        assert int(st) == R.MOE_STATUS_BAD_OFFSETS
        assert all(padding_kept(*v) for v in outs) and padding_kept(*dx)
    for of_two in (False, True):
        s = mx.make(sizes, 2568, 2048, seed=27, pad=16)
        s["off"] = off
        out, store = mx.strided(s["rows"], s["n"], BF16, 16)
        st = gated.status_word()
        mx.run(s, of_two, out, st)
        torch.cuda.synchronize()
        assert int(st) == R.MOE_STATUS_BAD_OFFSETS and padding_kept(out, store)


@pytest.mark.parametrize("way", gated.WAYS)
def test_repeated_and_on_two_streams(way):
    """The same bits every time, with another call of the largest tiles beside it."""
    n, k = WIDTHS[way]
    s = gated.make([500, 270, 2700, 900], n, k, BF16, seed=28)
    outs = [[torch.empty((s["rows"], n if way != "input" else k), dtype=BF16, device="cuda") for _ in range(3)] for _ in range(3)]

    def run(out, stream=None):
        if way == "forward":
            R.gated_forward(s["plan"], s["x"], s["w_gate"], s["w_up"], s["off"], *out, stream=stream)
        elif way == "hidden":
            R.gated_backward_h(s["plan"], s["dy"], s["w_down"], s["gate"], s["up"], s["off"], *out, stream=stream)
        else:
            R.gated_backward_x(s["plan"], s["dgate"], s["dup"], s["w_gate"], s["w_up"], s["off"], out[0], stream=stream)

    run(outs[0])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for out, stream in zip(outs[1:], streams):
            run(out, stream)
    torch.cuda.synchronize()
    for out in outs[1:]:
        for a, b in zip(out[:1 if way == "input" else 3], outs[0]):
            assert torch.equal(a, b)


def test_weights_past_32_bits():
    """Groups of 16-bit weights whose element offsets pass 2^31 and byte offsets 2^32, small and large tiles."""
    apart = (1 << 31) + 64
    store = torch.zeros(apart + 2568 * 1024, dtype=BF16, device="cuda")
    for sizes, width in (([9, 20], 136), ([1500, 2900], 2568)):
        s = gated.make(sizes, 1024, width, BF16, seed=29)
        for key in ("w_gate", "w_up"):
            dense = s[key].view(2, 1024, width)
            far = torch.as_strided(store, (2, 1024, width), (apart, width, 1))
            far.copy_(dense)
            plan = R.Gated(2, 1024, width, BF16, act=s["act"], limit=s["limit"], w_group_stride=apart)   # (as the other call)
            got, want = (torch.empty((s["rows"], width), dtype=BF16, device="cuda") for _ in range(2))
            R.gated_backward_x(plan, s["dgate"], s["dup"], far, far, s["off"], got)
            R.gated_backward_x(s["plan"], s["dgate"], s["dup"], dense, dense, s["off"], want)
            assert torch.equal(got, want)
            got, want = (torch.empty((s["rows"], 1024), dtype=BF16, device="cuda") for _ in range(2))
            R.gated_forward(plan, s["x"], far, far, s["off"], got)
            R.gated_forward(s["plan"], s["x"], dense, dense, s["off"], want)
            assert torch.equal(got, want)
