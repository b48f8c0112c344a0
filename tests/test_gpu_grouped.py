"""moe_grouped_* against the products in 64 bits.

Tolerances. Products of 16-bit values are exact in f32. A matrix instruction
sums 32 of them and adds them to the running sum: a term passes at most
32 + r / 32 + 1 additions for r terms, each off by at most 2^-23 of the sum of
the absolute terms (whether it rounds or truncates), then one rounding to the
output's type, half a step relative to the value (fp16: at least half its
smallest step)."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests.block_helpers import BF16, CANARY, F32, FP16, assert_within, fill, half_step, padding_kept, strided

pytestmark = pytest.mark.gpu

WAYS = ["forward", "dx", "dw"]


def bounds(sizes, first=0):
    out = [first]
    for v in sizes:
        out.append(out[-1] + v)
    return out


def make(sizes, n, k, t, seed, pad=0, offset=0, before=0, after=0):
    """Operands with rows of no group before and after the groups'; weights of different rows and groups apart by pad."""
    g = torch.Generator().manual_seed(seed)
    rows = before + sum(sizes) + after
    s = {"ends": bounds(sizes, before), "rows": rows, "n": n, "k": k, "t": t, "pad": pad, "offset": offset}
    s["off"] = torch.tensor(s["ends"], dtype=torch.int32, device="cuda")
    s["x"] = fill(strided(rows, k, t, pad, offset)[0], torch.randn((rows, k), generator=g))
    s["dy"] = fill(strided(rows, n, t, pad, offset)[0], torch.randn((rows, n), generator=g))
    w, _ = strided(len(sizes) * n, k, t, pad, offset)
    s["w"] = fill(w, torch.randn((len(sizes) * n, k), generator=g))
    return s


def plan(s, out):
    n, k, pad = s["n"], s["k"], s["pad"]
    return R.Grouped(len(s["ends"]) - 1, n, k, s["t"], out=out, x_stride=k + pad, y_stride=n + pad, w_stride=k + pad)


def want(s, way):
    """(value, sum of absolute terms, number of terms)."""
    n, k, ends = s["n"], s["k"], s["ends"]
    x, dy, w = s["x"].double(), s["dy"].double(), s["w"].double().reshape(-1, n, k)
    groups = len(ends) - 1
    shape = {"forward": (s["rows"], n), "dx": (s["rows"], k), "dw": (groups * n, k)}[way]
    v, mag = (torch.zeros(shape, dtype=torch.float64, device=x.device) for _ in range(2))
    most = {"forward": k, "dx": n, "dw": max(b - a for a, b in zip(ends, ends[1:]))}[way]
    for g in range(groups):
        a, b = ends[g], ends[g + 1]
        if a == b:
            continue
        if way == "forward":
            v[a:b], mag[a:b] = x[a:b] @ w[g].t().contiguous(), x[a:b].abs() @ w[g].abs().t().contiguous()
        elif way == "dx":
            v[a:b], mag[a:b] = dy[a:b] @ w[g], dy[a:b].abs() @ w[g].abs()
        else:
            r = slice(g * n, g * n + n)
            dyt = dy[a:b].t().contiguous()
            v[r], mag[r] = dyt @ x[a:b], dyt.abs() @ x[a:b].abs()
    return v, mag, most


def call(s, way, out, status=None, p=None):
    p = p or plan(s, out.dtype)
    if way == "forward":
        R.grouped_forward(p, s["x"], s["w"], s["off"], out, status)
    elif way == "dx":
        R.grouped_backward_x(p, s["dy"], s["w"], s["off"], out, status)
    else:
        R.grouped_backward_w(p, s["dy"], s["x"], s["off"], out, status)


def output(s, way, out):
    rows, cols = {"forward": (s["rows"], s["n"]), "dx": (s["rows"], s["k"]),
                  "dw": ((len(s["ends"]) - 1) * s["n"], s["k"])}[way]
    return strided(rows, cols, out, s["pad"], s["offset"] if out != F32 else s["offset"])


def tolerance(v, mag, most, out):
    return half_step(out) * v.abs() + (most / 32 + 33) * 2.0 ** -23 * mag + 1e-30 + (2.0 ** -25 if out == FP16 else 0.0)


def check(s, way, out):
    y, store = output(s, way, out)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(s, way, y, status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert padding_kept(y, store), "wrote outside its rows"
    v, mag, most = want(s, way)
    assert_within(y, v, tolerance(v, mag, most, out), f"{way} {s['t']} {s['n']}x{s['k']} {s['ends']}")
    return y


FEW = [0, 1, 3, 0, 0, 17, 2, 16, 1, 0, 5, 0]
SOME = [0, 40, 65, 1, 64, 63, 0, 33]
MANY = [130, 0, 128, 257, 1, 90]


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("n,k", [(64, 64), (128, 128), (136, 72), (8, 200), (264, 1000), (192, 320)])
@pytest.mark.parametrize("t", [BF16, FP16], ids=["bf16", "fp16"])
def test_aligned(way, n, k, t):
    for i, sizes in enumerate((FEW, SOME, MANY)):
        for out in (t, F32):
            check(make(sizes, n, k, t, seed=i, pad=8 * i, offset=8 * i, before=i, after=2 * i), way, out)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("n,k", [(1, 1), (1, 64), (64, 1), (7, 200), (257, 515), (129, 127), (65, 31)])
@pytest.mark.parametrize("t", [BF16, FP16], ids=["bf16", "fp16"])
def test_any_width_and_alignment(way, n, k, t):
    for i, sizes in enumerate((FEW, SOME, MANY)):
        check(make(sizes, n, k, t, seed=i, before=5 * i, after=i), way, t if i else F32)
    check(make(SOME, n, k, t, seed=9, pad=3, offset=1), way, F32)
    check(make(FEW, n, k, t, seed=9, pad=1, offset=5), way, t)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("pad,offset", [(8, 4), (4, 8), (2, 2), (0, 8)])
def test_alignment_between(way, pad, offset):
    """Rows of 8-, 4- and 16-byte alignment at widths that are multiples of 8."""
    check(make(SOME, 128, 192, BF16, seed=1, pad=pad, offset=offset), way, BF16)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("sizes", [[1], [0], [0, 0, 7], [300], [64] * 16, [1] * 700, [0] * 500 + [3] + [0] * 523,
                                   [2, 0] * 512, [4000], [4000, 1]], ids=lambda v: f"{len(v)}x{sum(v)}")
def test_groups(way, sizes):
    check(make(sizes, 64, 128, BF16, seed=2, before=1, after=3), way, BF16)
    check(make(sizes, 40, 24, FP16, seed=3), way, F32) if sum(sizes) else None


@pytest.mark.parametrize("way", WAYS)
def test_long_sums(way):
    """Sums over 4096 (the rows of one group, for the weights' gradient)."""
    n, k = {"forward": (192, 4096), "dx": (4096, 192), "dw": (192, 320)}[way]
    check(make([5, 4096, 100] if way == "dw" else [70, 0, 9], n, k, BF16, seed=4), way, F32)


def test_no_rows():
    s = make([0, 0, 0], 64, 72, BF16, seed=0)
    dw = torch.full((3 * 64, 72), CANARY, dtype=F32, device="cuda")
    call(s, "dw", dw)
    assert not dw.any()
    for way in ("forward", "dx"):
        y = torch.full((4, 72), CANARY, dtype=BF16, device="cuda")
        call(s, way, y)
        assert (y == CANARY).all()


@pytest.mark.parametrize("n,k", [(128, 128), (65, 67)])
def test_infinities_stay_in_their_group(n, k):
    """NaN and infinities in the rows or the weight of one group, and in rows of none, change no other group."""
    sizes = [20, 37, 5, 0, 70]
    a, b = 20, 57
    for way in WAYS:
        s = make(sizes, n, k, BF16, seed=6, before=2, after=4)
        a, b = s["ends"][1], s["ends"][2]
        clean, _ = output(s, way, BF16)
        call(s, way, clean)
        for v in (s["x"], s["dy"]):
            v[:2], v[-4:] = float("nan"), float("inf")
            v[a:b] = float("nan")
        s["w"][n:2 * n] = float("inf")
        y, _ = output(s, way, BF16)
        call(s, way, y)
        mine = slice(a, b) if way != "dw" else slice(n, 2 * n)
        assert y[mine].isnan().all()
        y[mine] = clean[mine]
        assert torch.equal(y, clean), way


@pytest.mark.parametrize("way", WAYS)
def test_bad_offsets_are_reported(way):
    """Offsets that descend or leave the rows: the status says so, and nothing outside the output is written."""
    for ends in ([0, 50, 20, 100], [-5, 10, 60, 100], [0, 10, 200, 100], [0, 2 ** 31 - 1, -2 ** 31, 70],
                 [100, 50, 20, 0]):
        s = make([40, 30, 30], 72, 64, BF16, seed=7, pad=8, offset=8)
        s["off"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        y, store = output(s, way, BF16)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(s, way, y, status)
        torch.cuda.synchronize()
        assert int(status) == R.MOE_STATUS_BAD_OFFSETS
        assert padding_kept(y, store)


def test_positions_past_32_bits():
    """Weights and rows whose element offsets pass 2^31."""
    n, k, groups, apart = 64, 128, 3, 2 ** 30 + 64
    s = make([40, 1, 30], n, k, BF16, seed=11)
    big = torch.zeros((groups - 1) * apart + n * k, dtype=BF16, device="cuda")
    view = torch.as_strided(big, (groups, n, k), (apart, k, 1))
    view.copy_(s["w"].view(groups, n, k))
    p = R.Grouped(groups, n, k, BF16, out=F32, w_group_stride=apart)
    for way, src in (("forward", s["x"]), ("dx", s["dy"])):
        y, _ = output(s, way, F32)
        (R.grouped_forward if way == "forward" else R.grouped_backward_x)(p, src, big, s["off"], y)
        v, mag, most = want(s, way)
        assert_within(y, v, tolerance(v, mag, most, F32), way)
    p = R.Grouped(groups, n, k, BF16, w_group_stride=apart)
    R.grouped_backward_w(p, s["dy"], s["x"], s["off"], big)
    v, mag, most = want(s, "dw")
    assert_within(view.reshape(groups * n, k), v, tolerance(v, mag, most, BF16), "dw")
    del big, view
    rows, stride = 1100, R.MOE_GROUPED_MAX_STRIDE
    s = make([500, 600], n, k, BF16, seed=12)
    big = torch.zeros((rows - 1) * stride + max(n, k), dtype=BF16, device="cuda")
    for way in WAYS:
        src, width = (s["dy"], n) if way == "dx" else (s["x"], k)
        view = torch.as_strided(big, (rows, width), (stride, 1))
        view.copy_(src)
        wide = {"x_stride": stride} if way != "dx" else {"y_stride": stride}
        p = R.Grouped(2, n, k, BF16, out=F32, **wide)
        y, _ = output(s, way, F32)
        if way == "forward":
            R.grouped_forward(p, view, s["w"], s["off"], y)
        elif way == "dx":
            R.grouped_backward_x(p, view, s["w"], s["off"], y)
        else:
            R.grouped_backward_w(p, s["dy"], view, s["off"], y)
        v, mag, most = want(s, way)
        assert_within(y, v, tolerance(v, mag, most, F32), way)


def test_gradients_against_differences():
    """The loss sum(dy y) is linear in x and in w: its differences along a direction are exact in 64 bits."""
    s = make([3, 0, 20, 9], 72, 40, FP16, seed=13)
    n, k, ends = 72, 40, s["ends"]
    x, w, dy = s["x"].double().cpu(), s["w"].double().cpu().view(-1, n, k), s["dy"].double().cpu()

    def loss(x, w):
        return sum(float((dy[a:b] * (x[a:b] @ w[g].t())).sum()) for g, (a, b) in enumerate(zip(ends, ends[1:])))

    dx, _ = output(s, "dx", F32)
    dw, _ = output(s, "dw", F32)
    call(s, "dx", dx)
    call(s, "dw", dw)
    gen = torch.Generator().manual_seed(1)
    for _ in range(3):
        v = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        u = torch.randn(w.shape, generator=gen, dtype=torch.float64)
        for got, slope in ((dx.double().cpu() * v, loss(x + v, w) - loss(x, w)),
                           (dw.double().cpu().view(w.shape) * u, loss(x, w + u) - loss(x, w))):
            # f32 gradients: (33 + 3) * 2^-23 of sums of at most 72 terms, whose absolute sums are below 72 * 16
            tol = 36 * 2.0 ** -23 * 72 * 16 * float((got != 0).sum()) ** 0.5 * 4 + 1e-9 * float(got.abs().sum())
            assert abs(float(got.sum()) - slope) <= tol


def test_other_stream_and_graph_replays():
    s = make(SOME, 136, 264, BF16, seed=21)
    first = {way: output(s, way, BF16)[0] for way in WAYS}
    again = {way: output(s, way, BF16)[0] for way in WAYS}
    for way in WAYS:
        call(s, way, first[way])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for way in WAYS:
            call(s, way, again[way])
    torch.cuda.synchronize()
    assert all(torch.equal(first[w], again[w]) for w in WAYS)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for way in WAYS:
            call(s, way, again[way])
    for _ in range(4):
        for v in again.values():
            v.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(first[w], again[w]) for w in WAYS)
        (torch.ones(1000, device="cuda") * 2).sum().item()
    # the replay reads the offsets of its time
    s["off"].copy_(torch.tensor([0] * len(SOME) + [sum(SOME)], dtype=torch.int32))
    s["ends"] = s["off"].tolist()
    graph.replay()
    v, mag, most = want(s, "dw")
    assert_within(again["dw"], v, tolerance(v, mag, most, BF16), "dw after new offsets")
