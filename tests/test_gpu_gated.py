"""moe_gated_* against the formulas in 64 bits.

Tolerances. The sums are those of the grouped products (see there): off by at
most (r / 32 + 33) 2^-23 of the sum of the absolute terms for r terms. An error e
of g moves act(g) by at most 1.2 e, clamps move nothing apart; the activation's
own error is in gated_helpers. Each output takes one more rounding of half a
step (fp16: at least half its smallest step)."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests.block_helpers import BF16, CANARY, F32, FP16, assert_within, fill, half_step, padding_kept, strided
from tests.gated_helpers import ACT, SLOPE, STEEPEST, activation, gradients, hidden, limited
from tests.test_gpu_grouped import FEW, MANY, SOME, bounds

pytestmark = pytest.mark.gpu


def make(sizes, n, k, t, seed=0, pad=0, offset=0, before=0, after=0, act="silu", limit=1.0, dx=None, sigma=None):
    gen = torch.Generator().manual_seed(seed)
    rows, groups = before + sum(sizes) + after, len(sizes)
    s = {"ends": bounds(sizes, before), "rows": rows, "groups": groups, "n": n, "k": k, "t": t, "pad": pad,
         "offset": offset, "act": act, "limit": limit, "dx": dx or t}
    s["off"] = torch.tensor(s["ends"], dtype=torch.int32, device="cuda")

    def filled(rows, cols, scale=1.0):
        return fill(strided(rows, cols, t, pad, offset)[0], torch.randn((rows, cols), generator=gen) * scale)

    s["x"], s["dy"] = filled(rows, k), filled(rows, k)
    s["w_gate"], s["w_up"] = (filled(groups * n, k, sigma or 1.5 * k ** -0.5) for _ in range(2))
    s["w_down"] = filled(groups * k, n, k ** -0.5)
    s["gate"], s["up"], s["dgate"], s["dup"] = (filled(rows, n, 1.5) for _ in range(4))
    s["plan"] = R.Gated(groups, n, k, t, act=act, limit=limit, dx=s["dx"], x_stride=k + pad, h_stride=n + pad,
                        gate_stride=n + pad, y_stride=k + pad, w_stride=k + pad, down_stride=n + pad)
    return s


def by_group(s, out, f):
    for g, (a, b) in enumerate(zip(s["ends"], s["ends"][1:])):
        if a < b:
            out[a:b] = f(g, a, b)
    return out


def zeros(s, cols):
    return torch.zeros((s["rows"], cols), dtype=torch.float64, device="cuda")


def weight(s, key):
    rows = s["k"] if key == "w_down" else s["n"]
    return s[key].double().reshape(s["groups"], rows, -1)


def sums(s, v, key, way):
    """The products of v's rows with the group's weight (way "t": its transpose) and the error of their f32 sums."""
    w, v = weight(s, key), v.double()
    cols, most = (w.shape[2], w.shape[1]) if way == "t" else (w.shape[1], w.shape[2])

    def product(v, w):
        return by_group(s, zeros(s, cols), lambda g, a, b: v[a:b] @ (w[g] if way == "t" else w[g].t().contiguous()))

    return product(v, w), (most / 32 + 33) * 2.0 ** -23 * product(v.abs(), w.abs())


def rounded(v, t):
    return half_step(t) * v.abs() + (2.0 ** -25 if t == FP16 else 2.0 ** -130)


def output(s, cols, t):
    return strided(s["rows"], cols, t, s["pad"], s["offset"])


def finish(s, outs, status):
    torch.cuda.synchronize()
    assert int(status) == 0
    for view, store in outs:
        assert padding_kept(view, store), "wrote outside its rows"


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def check_forward(s, kept=True):
    outs = [output(s, s["n"], s["t"]) for _ in range(3 if kept else 1)]
    st = status_word()
    R.gated_forward(s["plan"], s["x"], s["w_gate"], s["w_up"], s["off"], *(v for v, _ in outs), status=st)
    finish(s, outs, st)
    (g, eg), (u, eu) = (sums(s, s["x"], key, "n") for key in ("w_gate", "w_up"))
    if kept:
        assert_within(outs[1][0], g, rounded(g, s["t"]) + 1.01 * eg, "gate")
        assert_within(outs[2][0], u, rounded(u, s["t"]) + 1.01 * eu, "up")
    gc, uc = limited(g, u, s["limit"])
    a = activation(gc, s["act"])[0]
    off = STEEPEST * eg + ACT * (gc.abs() + eg)
    h = a * uc
    tol = rounded(h, s["t"]) + 1.01 * (off * (uc.abs() + eu) + a.abs() * eu) + 2.0 ** -22 * h.abs()
    assert_within(outs[0][0], h, tol, f"h {s['t']} {s['n']}x{s['k']} {s['ends']}")
    return [v for v, _ in outs]


def check_hidden(s, again=True, in_place=False):
    outs = [output(s, s["n"], s["t"]) for _ in range(3)]
    (dgate, _), (dup, _), (h, _) = outs
    g, u = s["gate"].double(), s["up"].double()
    gate, up = s["gate"], s["up"]
    if in_place:
        fill(dgate, gate)
        fill(dup, up)
        gate, up = dgate, dup
    st = status_word()
    R.gated_backward_h(s["plan"], s["dy"], s["w_down"], gate, up, s["off"], dgate, dup, h if again else None, status=st)
    finish(s, outs, st)
    if not again:
        assert (h == CANARY).all()
    dh, e = sums(s, s["dy"], "w_down", "t")
    inside = torch.zeros((s["rows"], 1), dtype=torch.bool, device="cuda")
    inside[s["ends"][0]:s["ends"][-1]] = True
    gc, uc = limited(g, u, s["limit"])
    a, slope = activation(gc, s["act"])
    dg, du = gradients(g, u, dh, s["act"], s["limit"])
    e2 = 1.01 * (e + 2.0 ** -22 * dh.abs())
    big = dh.abs() + e2
    assert_within(dgate, dg, rounded(dg, s["t"]) + 1.01 * uc.abs() * (e2 * slope.abs() + big * SLOPE), "dgate")
    assert_within(dup, du, rounded(du, s["t"]) + 1.01 * (e2 * a.abs() + big * ACT * gc.abs()), "dup")
    if again:
        want = torch.where(inside, a * uc, 0.0)
        assert_within(h, want, rounded(want, s["t"]) + 1.01 * ACT * gc.abs() * uc.abs(), "h")
    return dgate, dup, h


def check_input(s):
    dx, store = output(s, s["k"], s["dx"])
    st = status_word()
    R.gated_backward_x(s["plan"], s["dgate"], s["dup"], s["w_gate"], s["w_up"], s["off"], dx, status=st)
    finish(s, [(dx, store)], st)
    (a, ea), (b, eb) = sums(s, s["dgate"], "w_gate", "t"), sums(s, s["dup"], "w_up", "t")
    # one running sum over both: each term passes the additions of both
    assert_within(dx, a + b, rounded(a + b, s["dx"]) + 2.02 * (ea + eb), f"dx {s['t']} {s['n']}x{s['k']} {s['ends']}")
    return dx


CHECKS = {"forward": check_forward, "hidden": check_hidden, "input": check_input}
WAYS = list(CHECKS)
TYPES = pytest.mark.parametrize("t", [BF16, FP16], ids=["bf16", "fp16"])


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("n,k", [(64, 64), (128, 128), (136, 72), (8, 200), (264, 1000), (192, 320)])
@TYPES
def test_aligned(way, n, k, t):
    for i, sizes in enumerate((FEW, SOME, MANY)):
        CHECKS[way](make(sizes, n, k, t, seed=i, pad=8 * i, offset=8 * i, before=i, after=2 * i,
                         act=("silu", "gelu")[i % 2], limit=(0.0, 1.0, 0.5)[i], dx=(F32, t)[i % 2]))


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("n,k", [(1, 1), (1, 64), (64, 1), (7, 200), (257, 515), (129, 127), (65, 31), (17, 16)])
@TYPES
def test_any_width_and_alignment(way, n, k, t):
    for i, sizes in enumerate((FEW, SOME, MANY)):
        CHECKS[way](make(sizes, n, k, t, seed=i, before=5 * i, after=i, act=("gelu", "silu")[i % 2]))
    CHECKS[way](make(SOME, n, k, t, seed=9, pad=3, offset=1, limit=0.0, dx=F32))
    CHECKS[way](make(FEW, n, k, t, seed=9, pad=1, offset=5))


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("sizes", [[1], [0], [0, 0, 7], [300], [64] * 16, [1] * 700, [0] * 500 + [3] + [0] * 523,
                                   [2, 0] * 512, [4000], [4000, 1]], ids=lambda v: f"{len(v)}x{sum(v)}")
def test_groups(way, sizes):
    CHECKS[way](make(sizes, 64, 128, BF16, seed=2, before=1, after=3))
    if sum(sizes):
        CHECKS[way](make(sizes, 40, 24, FP16, seed=3))


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("sizes,n,k", [([700, 0, 900, 450], 1024, 1088), ([2100, 1900, 1, 2100], 2048, 1152),
                                       ([3000], 2056, 1032)], ids=["4 groups", "large tiles", "one group"])
def test_large_tiles(way, sizes, n, k):
    CHECKS[way](make(sizes, n, k, BF16, seed=4, before=2, after=1))


@pytest.mark.parametrize("way", WAYS)
def test_long_sums(way):
    CHECKS[way](make([3, 20], 8192 if way == "input" else 72, 72 if way == "input" else 16384, BF16, seed=5))


def test_without_what_may_be_left_out():
    s = make(SOME, 136, 200, BF16, seed=6)
    h = check_forward(s)[0]
    assert torch.equal(h, check_forward(s, kept=False)[0])
    a = check_hidden(s)
    b = check_hidden(s, again=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n,k", [(136, 200), (129, 61)])
def test_gradients_in_place(n, k):
    s = make(SOME, n, k, FP16, seed=7, before=2)
    for a, b in zip(check_hidden(s), check_hidden(s, in_place=True)):
        assert torch.equal(a, b)


def test_weights_and_gates_in_one_tensor():
    """Halves of a stacked weight and of rows of 2 n, in either order, as views."""
    s = make(SOME, 64, 96, BF16, seed=8)
    g, n, k, rows = s["groups"], 64, 96, s["rows"]
    want_h, want_gate, want_up = check_forward(s)
    dx = check_input(s)
    for swap in (False, True):
        w = torch.empty((g, 2, n, k), dtype=BF16, device="cuda")
        w[:, int(swap)], w[:, 1 - int(swap)] = weight(s, "w_gate").to(BF16), weight(s, "w_up").to(BF16)
        p = R.Gated(g, n, k, BF16, limit=1.0, gate_stride=2 * n, w_group_stride=2 * n * k)
        gu = torch.full((rows, 2 * n), 5.0, dtype=BF16, device="cuda")
        h = torch.empty((rows, n), dtype=BF16, device="cuda")
        gate, up = (gu[:, n:], gu[:, :n]) if swap else (gu[:, :n], gu[:, n:])
        R.gated_forward(p, s["x"], w[:, int(swap)], w[:, 1 - int(swap)], s["off"], h, gate, up)
        assert torch.equal(h, want_h) and torch.equal(gate, want_gate) and torch.equal(up, want_up)
        gate.copy_(s["dgate"])
        up.copy_(s["dup"])
        got = torch.empty((rows, k), dtype=BF16, device="cuda")
        R.gated_backward_x(p, gate, up, w[:, int(swap)], w[:, 1 - int(swap)], s["off"], got)
        assert torch.equal(got, dx)


@TYPES
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_values_at_the_ends(t, act):
    """Large, infinite and NaN products: the limits' values where a clamp holds them, NaN where there is one."""
    big = 60000.0
    values = torch.tensor([0.0, -0.0, 1.0, -1.0, 9.0, -9.0, 50.0, -50.0, 90.0, -90.0, 120.0, -120.0, big, -big,
                           float("inf"), -float("inf"), float("nan"), 1e-7], dtype=F32)
    m = values.numel()
    off = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    x = torch.zeros((m, 8), dtype=t, device="cuda")
    x[:, 0] = values.to(t)
    w = torch.zeros((m, 8), dtype=t, device="cuda")
    w[:, 0] = 1.0
    one = torch.zeros((m, 8), dtype=t, device="cuda")
    one[:, 0] = 1.0
    for limit in (0.0, 7.0):
        # x's value through the gate, with an up product of 1 (row 0 of each is 1 x value)
        p = R.Gated(1, m, 8, t, act=act, limit=limit)
        h, gate, up = (torch.empty((m, m), dtype=t, device="cuda") for _ in range(3))
        R.gated_forward(p, x, w, w, off, h, gate, up)
        v = x[:, 0].double()
        fin = v.isfinite()
        want = hidden(v, v, act, limit)
        if limit or t == BF16:   # (60000 squared is past fp16)
            assert_within(h[fin, 0], want[fin], rounded(want[fin], t) + 2.0 ** -17 * want[fin].abs() + 2.0 ** -19, "h")
        assert h[16].isnan().all()
        if limit:   # +inf is held by both clamps; -inf only by up's, where act is 0
            assert_within(h[14, :1], hidden(torch.full((1,), 7.0, dtype=torch.float64, device="cuda"),
                                            torch.full((1,), 7.0, dtype=torch.float64, device="cuda"), act, 0.0),
                          torch.full((1,), 49.0 * half_step(t) * 1.01, device="cuda"), "h of inf")
            assert (h[15, 0] == 0).all()
        # the gradients: dh = 1 in every column
        gate.copy_(v[:, None].expand(m, m).to(t))
        up.copy_(v[None, :].expand(m, m).to(t))
        dg, du, again = (torch.empty((m, m), dtype=t, device="cuda") for _ in range(3))
        R.gated_backward_h(p, one, torch.ones((8, m), dtype=t, device="cuda"), gate, up, off, dg, du, again)
        gd, ud = gate.double(), up.double()
        wg, wu = gradients(gd, ud, torch.ones_like(gd), act, limit)
        both = gd.isfinite() & ud.isfinite()
        ok = both & (wg.abs() < torch.finfo(t).max / 2) & (wu.abs() < torch.finfo(t).max / 2)
        assert_within(dg[ok], wg[ok], rounded(wg[ok], t) + SLOPE * limited(gd, ud, limit)[1].abs()[ok] * 2, "dgate")
        assert_within(du[ok], wu[ok], rounded(wu[ok], t) + ACT * gd.abs()[ok] * 2, "dup")
        if limit:
            assert (dg[14] == 0)[:16].all() and (du[:, 14] == 0)[:16].all() and (du[:, 15] == 0)[:16].all()
        assert dg[16, 2].isnan() and du[16, 2].isnan() and dg[2, 16].isnan()


def test_gradients_against_differences():
    """The kernels' gradients against central differences of the kernels' own forward pass in what it sums."""
    s = make([5, 9], 24, 40, FP16, seed=10, act="gelu", limit=2.0)
    g, u = (sums(s, s["x"], key, "n")[0] for key in ("w_gate", "w_up"))
    dh = sums(s, s["dy"], "w_down", "t")[0]
    s["gate"].copy_(g)
    s["up"].copy_(u)
    dgate, dup, _ = check_hidden(s)
    gk, uk, step = s["gate"].double(), s["up"].double(), 1e-4
    clear = ((gk - 2).abs() > 1e-3) & ((uk.abs() - 2).abs() > 1e-3)   # the clamps' corners have no slope
    for got, d in ((dgate, (hidden(gk + step, uk, "gelu", 2.0) - hidden(gk - step, uk, "gelu", 2.0)) / (2 * step)),
                   (dup, (hidden(gk, uk + step, "gelu", 2.0) - hidden(gk, uk - step, "gelu", 2.0)) / (2 * step))):
        want = dh * d
        # the differences are off by step^2 / 6 of the third derivative (below 4), the kernel by its tolerance
        tol = rounded(want, FP16) + 1e-7 * dh.abs() + 2.0 ** -12 * dh.abs() * (1 + uk.abs() + gk.abs())
        assert_within(got[clear], want[clear], tol[clear], "difference")


def test_whole_block_against_autograd():
    """Forward, then all gradients of a block as a training step calls them, against autograd in 64 bits. The gradients are
    those at the kept gate and up: a product within half a step of a clamp's end may lie on its other side there, where
    the derivative jumps, so the oracle's activation is taken at the kept values too (passing gradients on unchanged)."""
    s = make([30, 0, 70, 5], 72, 104, BF16, seed=11, limit=1.5)
    n, k, groups, rows = s["n"], s["k"], s["groups"], s["rows"]
    h, gate, up = check_forward(s)
    y = torch.empty((rows, k), dtype=BF16, device="cuda")
    R.grouped_forward(R.Grouped(groups, k, n, BF16), h, s["w_down"], s["off"], y)
    dgate, dup, again = (torch.empty_like(h) for _ in range(3))
    R.gated_backward_h(s["plan"], s["dy"], s["w_down"], gate, up, s["off"], dgate, dup, again)
    dx = torch.empty_like(y)
    R.gated_backward_x(s["plan"], dgate, dup, s["w_gate"], s["w_up"], s["off"], dx)
    dw = {key: torch.empty((groups, n, k), dtype=F32, device="cuda") for key in ("w_gate", "w_up")}
    up_w = R.Grouped(groups, n, k, BF16, out=F32)
    R.grouped_backward_w(up_w, dgate, s["x"], s["off"], dw["w_gate"])
    R.grouped_backward_w(up_w, dup, s["x"], s["off"], dw["w_up"])
    dw["w_down"] = torch.empty((groups, k, n), dtype=F32, device="cuda")
    R.grouped_backward_w(R.Grouped(groups, k, n, BF16, out=F32), s["dy"], again, s["off"], dw["w_down"])
    leaves = {key: weight(s, key).requires_grad_() for key in dw}
    x = s["x"].double().requires_grad_()
    loss, ys = 0.0, []
    for e, (a, b) in enumerate(zip(s["ends"], s["ends"][1:])):
        g, u = x[a:b] @ leaves["w_gate"][e].t(), x[a:b] @ leaves["w_up"][e].t()
        v = hidden(g + (gate[a:b].double() - g).detach(), u + (up[a:b].double() - u).detach(), "silu", 1.5)
        ys.append(v @ leaves["w_down"][e].t())
        loss = loss + (ys[-1] * s["dy"][a:b].double()).sum()
    loss.backward()
    # at most four roundings to 16 bits lie between the inputs and any result, in norm
    for got, want, what in [(y, torch.cat(ys).detach(), "y"), (dx, x.grad, "dx")] + [
            (dw[key].double(), leaves[key].grad, key) for key in dw]:
        off = float((got.double() - want).norm() / want.norm())
        assert off <= 4 * half_step(BF16), f"{what}: {off:.3g}"


@pytest.mark.parametrize("way", WAYS)
def test_captured_and_replayed(way):
    """Replays of one captured call, with new inputs and eager work between them, give the eager call's bits."""
    s = make(MANY, 136, 264, BF16, seed=12)
    n, rows = s["n"], s["rows"]
    outs = [torch.empty((rows, n), dtype=BF16, device="cuda") for _ in range(3)]
    dx = torch.empty((rows, s["k"]), dtype=BF16, device="cuda")

    def call(outs, dx):
        if way == "forward":
            R.gated_forward(s["plan"], s["x"], s["w_gate"], s["w_up"], s["off"], *outs)
        elif way == "hidden":
            R.gated_backward_h(s["plan"], s["dy"], s["w_down"], s["gate"], s["up"], s["off"], *outs)
        else:
            R.gated_backward_x(s["plan"], s["dgate"], s["dup"], s["w_gate"], s["w_up"], s["off"], dx)

    call(outs, dx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs, dx)
    for i in range(4):
        for key in ("x", "dy", "gate", "up", "dgate", "dup"):
            s[key].mul_(-0.75)
        for v in (*outs, dx):
            v.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        eager, edx = [torch.empty_like(v) for v in outs], torch.empty_like(dx)
        call(eager, edx)
        got, want = ([dx], [edx]) if way == "input" else (outs, eager)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_on_a_stream_of_its_own_and_two_at_once():
    a, b = make(MANY, 136, 264, BF16, seed=13), make(SOME, 200, 136, BF16, seed=14)
    want = [check_forward(v, kept=False)[0] for v in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [torch.empty((v["rows"], v["n"]), dtype=BF16, device="cuda") for v in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        for v, h, stream in zip((a, b), got, streams):
            R.gated_forward(v["plan"], v["x"], v["w_gate"], v["w_up"], v["off"], h, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("ends", [[0, 5, 3, 9], [0, 4, 9, 13], [-2, 4, 6, 9], [9, 6, 3, 0], [1 << 30, 0, (1 << 31) - 1, 2]])
def test_bad_offsets_are_reported(ends):
    """Offsets that do not ascend inside [0, rows]: the status says so, and nothing outside the buffers changes."""
    s = make([3, 3, 3], 40, 48, BF16, seed=15, pad=8)
    off = torch.tensor([max(min(v, (1 << 31) - 1), -(1 << 31)) for v in ends], dtype=torch.int64).to(torch.int32).cuda()
    outs = [output(s, s["n"], BF16) for _ in range(3)]
    dx = output(s, s["k"], BF16)
    for call in (lambda st: R.gated_forward(s["plan"], s["x"], s["w_gate"], s["w_up"], off, *(v for v, _ in outs), status=st),
                 lambda st: R.gated_backward_h(s["plan"], s["dy"], s["w_down"], s["gate"], s["up"], off,
                                               *(v for v, _ in outs), status=st),
                 lambda st: R.gated_backward_x(s["plan"], s["dgate"], s["dup"], s["w_gate"], s["w_up"], off, dx[0],
                                               status=st)):
        st = status_word()
        call(st)
        torch.cuda.synchronize()
        assert int(st) == R.MOE_STATUS_BAD_OFFSETS
        assert all(padding_kept(*v) for v in outs) and padding_kept(*dx)


def test_no_rows():
    s = make([3, 2], 40, 48, BF16, seed=16)
    empty = torch.empty((0, 48), dtype=BF16, device="cuda")
    hidden_rows = torch.empty((0, 40), dtype=BF16, device="cuda")
    for ends, code in (([0, 0, 0], 0), ([0, 1, 2], R.MOE_STATUS_BAD_OFFSETS)):
        off = torch.tensor(ends, dtype=torch.int32, device="cuda")
        for call in (lambda st: R.gated_forward(s["plan"], empty, s["w_gate"], s["w_up"], off, hidden_rows, status=st),
                     lambda st: R.gated_backward_h(s["plan"], empty, s["w_down"], hidden_rows, hidden_rows, off, hidden_rows,
                                                   hidden_rows, status=st),
                     lambda st: R.gated_backward_x(s["plan"], hidden_rows, hidden_rows, s["w_gate"], s["w_up"], off, empty,
                                                   status=st)):
            st = status_word()
            call(st)
            torch.cuda.synchronize()
            assert int(st) == code
