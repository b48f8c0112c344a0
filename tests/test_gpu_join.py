"""moe_join_forward / moe_join_backward against the formulas in 64 bits.

Tolerances. One output rounding is half a step of its type, relative to the
value. Before it everything is f32: a row's sum of up to 16384 terms passes at
most 48 roundings on the way of any term (16 in a thread, 6 in a wave, 16 over
the waves, and the products), the norm takes half of its relative error plus
three roundings, and each value a handful more: together below 2^-18 of the
sum of the absolute values of the terms that make the value (2^-17 for what
passes two such sums). A sum over m rows adds at most m / 512 + 128 + 4
roundings of 2^-24 of the sum of the absolute terms."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests.block_helpers import BF16, F32, FP16, assert_within, fill, half_step, padding_kept, strided

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make(m, dim, t, res, gate, post, seed, pad=0, offset=0):
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape, mean=0.0, sigma=1.0):
        return torch.randn(shape, generator=g, dtype=torch.float64) * sigma + mean

    def put(dtype, values):
        v, store = strided(*values.shape, dtype, pad, offset)
        return fill(v, values), store

    s = {}
    s["x"], s["x_store"] = put(res, rnd(m, dim, sigma=2.0))
    s["b"], s["b_store"] = put(t, rnd(m, dim))
    s["w_pre"] = rnd(dim, mean=1.0, sigma=0.3).to(t).cuda()
    s["w_post"] = rnd(dim, mean=1.0, sigma=0.3).to(t).cuda() if post else None
    s["gate"] = None
    if gate == "shared":
        s["gate"] = rnd(dim, mean=0.5, sigma=0.5).to(t).cuda()
    elif gate == "rows":
        s["gate"], s["gate_store"] = put(t, rnd(m, dim, mean=0.5, sigma=0.5))
    s["dy"], _ = put(t, rnd(m, dim))
    s["dxo"], _ = put(res, rnd(m, dim))
    st = dim + pad
    s["plan"] = R.Join(dim, t, residual=res, gate_rows=gate == "rows", scale=0.7, eps=EPS, x_stride=st,
                       x_out_stride=st, b_stride=st, gate_stride=st, y_stride=st)
    return s


def d(v):
    return None if v is None else v.double().cpu()


def formulas(s, x_out=None):
    """(outputs, magnitudes) of the forward pass, and of the gradients where the stored stream is given."""
    scale = float(torch.tensor(0.7, dtype=torch.float32))
    eps = float(torch.tensor(EPS, dtype=torch.float32))
    x, b, w_pre, w_post = d(s["x"]), d(s["b"]), d(s["w_pre"]), d(s["w_post"])
    gain = scale * (torch.ones_like(b) if s["gate"] is None else d(s["gate"]).expand_as(b))
    rb = (b.square().mean(1, keepdim=True) + eps).rsqrt() if w_post is not None else torch.ones_like(b[:, :1])
    nb = b * rb
    wp = w_post if w_post is not None else torch.ones(b.shape[1], dtype=torch.float64)
    z = nb * wp
    if x_out is None:
        xo = x + gain * z
        mag = x.abs() + (gain * z).abs()
        rx = (xo.square().mean(1, keepdim=True) + eps).rsqrt()
        return {"x_out": xo, "y": xo * rx * w_pre}, {"x_out": mag, "y": mag * rx * w_pre.abs()}
    xo, dy, dxo = d(x_out), d(s["dy"]), d(s["dxo"])
    rx = (xo.square().mean(1, keepdim=True) + eps).rsqrt()
    n, dn = xo * rx, dy * w_pre
    dx = dxo + rx * (dn - n * (dn * n).mean(1, keepdim=True))
    dx_m = dxo.abs() + rx * (dn.abs() + n.abs() * (dn * n).abs().mean(1, keepdim=True))
    dz, dz_m = gain * dx, gain.abs() * dx_m
    out = {"dx": dx, "dw_pre": (dy * n).sum(0)}
    mag = {"dx": dx_m, "dw_pre": (dy * n).abs().sum(0)}
    if w_post is not None:
        h, h_m = dz * wp, dz_m * wp.abs()
        out["db"] = rb * (h - nb * (h * nb).mean(1, keepdim=True))
        mag["db"] = rb * (h_m + nb.abs() * (h_m * nb.abs()).mean(1, keepdim=True))
        out["dw_post"], mag["dw_post"] = (dz * nb).sum(0), (dz_m * nb.abs()).sum(0)
    else:
        out["db"], mag["db"] = dz, dz_m
    if s["gate"] is not None:
        dg, dg_m = scale * dx * z, scale * dx_m * z.abs()
        rows = s["gate"].dim() == 2
        out["dgate"], mag["dgate"] = (dg, dg_m) if rows else (dg.sum(0), dg_m.sum(0))
    return out, mag


def forward(s, pad, offset, in_place=False):
    m, dim = s["x"].shape
    if in_place:
        x_out, y = s["x"], s["b"]
        R.join_forward(s["plan"], s["x"], s["b"], s["w_post"], s["gate"], s["w_pre"], x_out, y)
        return x_out, y
    x_out, xs = strided(m, dim, s["x"].dtype, pad, offset)
    y, ys = strided(m, dim, s["b"].dtype, pad, offset)
    R.join_forward(s["plan"], s["x"], s["b"], s["w_post"], s["gate"], s["w_pre"], x_out, y)
    torch.cuda.synchronize()
    assert padding_kept(x_out, xs) and padding_kept(y, ys)
    return x_out, y


def check_forward(s, x_out, y, want, mag):
    for name, got in (("x_out", x_out), ("y", y)):
        assert_within(got, want[name], half_step(got.dtype) * want[name].abs() + 2.0 ** -18 * mag[name] + 1e-30
                      + (2.0 ** -25 if got.dtype == FP16 else 0.0), name)   # (fp16: half its smallest step)


DIMS = [1, 7, 64, 511, 512, 513, 1001, 1024, 2048, 2050, 4096, 4099, 8192, 8200, 16384]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("t,res", [(BF16, BF16), (FP16, F32)], ids=["bf16", "fp16-f32"])
def test_forward_widths(dim, t, res):
    for m, gate, post, pad, offset in ((3, "shared", True, 0, 0), (5, "rows", False, 5, 3), (1, "none", True, 8, 8)):
        s = make(m, dim, t, res, gate, post, seed=dim + m, pad=pad, offset=offset)
        want, mag = formulas(s)
        x_out, y = forward(s, pad, offset)
        check_forward(s, x_out, y, want, mag)


@pytest.mark.parametrize("t,res", [(BF16, F32), (FP16, FP16)], ids=["bf16-f32", "fp16"])
def test_forward_many_rows_and_in_place(t, res):
    for m, dim in ((1000, 512), (777, 1001), (300, 4096)):
        s = make(m, dim, t, res, "shared", True, seed=m)
        want, mag = formulas(s)
        x_out, y = forward(s, 0, 0)
        check_forward(s, x_out, y, want, mag)
        xi, yi = forward(s, 0, 0, in_place=True)
        assert torch.equal(xi, x_out) and torch.equal(yi, y)


def test_parts_alone():
    """Only the norm of the stream (no block yet); only the residual add (no norm after it)."""
    s = make(9, 640, BF16, F32, "shared", True, seed=4)
    y = torch.empty((9, 640), dtype=BF16, device="cuda")
    R.join_forward(s["plan"], s["x"], None, None, None, s["w_pre"], None, y)
    x = d(s["x"])
    want = x * (x.square().mean(1, keepdim=True) + EPS).rsqrt() * d(s["w_pre"])
    assert_within(y, want, half_step(BF16) * want.abs() + 2.0 ** -18 * want.abs() + 1e-30, "y alone")
    x_out = torch.empty_like(s["x"])
    R.join_forward(s["plan"], s["x"], s["b"], s["w_post"], s["gate"], None, x_out, None)
    both, _ = forward(s, 0, 0)
    assert torch.equal(x_out, both)


def test_special_rows():
    """A zero row has zero norms and stays finite; an infinity or NaN stays in its own row."""
    for dim in (640, 4096):
        s = make(6, dim, BF16, F32, "none", True, seed=8)
        clean = forward(s, 0, 0)
        s["x"][1], s["b"][1] = 0.0, 0.0
        s["b"][3, 5] = float("inf")
        s["x"][4, 7] = float("nan")
        x_out, y = forward(s, 0, 0)
        assert not x_out[1].any() and not y[1].any()
        assert x_out[3].isnan().any() and y[3].isnan().any() and y[4].isnan().all()
        for row in (0, 2, 5):
            assert torch.equal(x_out[row], clean[0][row]) and torch.equal(y[row], clean[1][row])


def backward(s, x_out, pad=0, offset=0, want=("db", "dw_post", "dgate", "dw_pre")):
    m, dim = s["x"].shape
    t, res = s["b"].dtype, s["x"].dtype
    out = {"dx": strided(m, dim, res, pad, offset)}
    if "db" in want:
        out["db"] = strided(m, dim, t, pad, offset)
    vec = lambda: torch.full((dim + 2,), -77.0, dtype=F32, device="cuda")  # noqa: E731
    vecs = {}
    if "dw_pre" in want:
        vecs["dw_pre"] = vec()
    if "dw_post" in want and s["w_post"] is not None:
        vecs["dw_post"] = vec()
    if "dgate" in want and s["gate"] is not None:
        if s["gate"].dim() == 2:
            out["dgate"] = strided(m, dim, t, pad, offset)
        else:
            vecs["dgate"] = vec()
    ws = torch.empty(R.join_workspace_bytes(s["plan"], m), dtype=torch.uint8, device="cuda")
    get = {**{k: v[0] for k, v in out.items()}, **{k: v[:dim] for k, v in vecs.items()}}
    R.join_backward(s["plan"], s["dy"], s["dxo"], x_out, s["b"], s["w_post"], s["gate"], s["w_pre"], get["dx"],
                    get.get("db"), get.get("dw_post"), get.get("dgate"), get.get("dw_pre"), ws)
    torch.cuda.synchronize()
    for k, (v, store) in out.items():
        assert padding_kept(v, store), k
    assert all((v[dim:] == -77.0).all() for v in vecs.values())
    return get


def check_backward(s, got, want, mag):
    m = s["x"].shape[0]
    for name, v in got.items():
        tol = 2.0 ** -17 * mag[name] + 1e-30 + (2.0 ** -25 if v.dtype == FP16 else 0.0)
        if v.dim() == 2:
            tol = tol + half_step(v.dtype) * want[name].abs()
        else:
            tol = tol + (m / 512 + 133) * 2.0 ** -24 * mag[name]
        assert_within(v, want[name], tol, name)


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("t,res", [(BF16, F32), (FP16, FP16)], ids=["bf16-f32", "fp16"])
def test_backward_widths(dim, t, res):
    for m, gate, post, pad, offset in ((3, "shared", True, 0, 0), (5, "rows", True, 5, 3), (2, "none", False, 8, 8),
                                       (4, "shared", False, 1, 0)):
        s = make(m, dim, t, res, gate, post, seed=dim + m, pad=pad, offset=offset)
        x_out, _ = forward(s, pad, offset)
        want, mag = formulas(s, x_out)
        check_backward(s, backward(s, x_out, pad, offset), want, mag)


@pytest.mark.parametrize("m,dim", [(1, 4096), (513, 512), (1030, 1001), (600, 4096)])
def test_backward_many_rows(m, dim):
    s = make(m, dim, BF16, BF16, "shared", True, seed=m)
    x_out, _ = forward(s, 0, 0)
    want, mag = formulas(s, x_out)
    got = backward(s, x_out)
    check_backward(s, got, want, mag)
    again = backward(s, x_out)
    assert all(torch.equal(got[k], again[k]) for k in got)
    # parts of it alone give the same bits
    for names in (("db",), ("dw_pre",), ("dgate", "dw_post")):
        part = backward(s, x_out, want=names)
        assert all(torch.equal(part[k], got[k]) for k in part)


def test_backward_of_one_side():
    """No gradient at y, or none at the stream; in place."""
    s = make(40, 1024, BF16, F32, "shared", True, seed=3)
    x_out, _ = forward(s, 0, 0)
    full = dict(s)
    for gone in ("dy", "dxo"):
        s = dict(full)
        zero = dict(full)
        s[gone] = None
        zero[gone] = torch.zeros_like(full[gone])
        want, mag = formulas(zero, x_out)
        names = ("db", "dw_post", "dgate") + (("dw_pre",) if gone == "dxo" else ())
        check_backward(s, backward(s, x_out, want=names), want, mag)
    got = backward(full, x_out)
    ws = torch.empty(R.join_workspace_bytes(full["plan"], 40), dtype=torch.uint8, device="cuda")
    dx, db = full["dxo"].clone(), full["b"].clone()
    R.join_backward(full["plan"], full["dy"], dx, x_out, db, full["w_post"], full["gate"], full["w_pre"], dx, db,
                    None, None, None, ws)
    assert torch.equal(dx, got["dx"]) and torch.equal(db, got["db"])


@pytest.mark.parametrize("gate,post", [("shared", True), ("rows", True), ("none", False)])
def test_gradients_against_differences(gate, post):
    """The loss sum(dy y) + sum(dx_out x') along random directions, by central differences in 64 bits. The
    differences' own error is h^2 times a third derivative (h = 1e-4, all values of order one): below 1e-6 of the
    scale; the kernel's bf16 gradients carry half a step each."""
    m, dim = 3, 72
    s = make(m, dim, BF16, F32, gate, post, seed=17)
    x_out, _ = forward(s, 0, 0)
    got = backward(s, x_out)
    dy, dxo = d(s["dy"]), d(s["dxo"])
    base = {k: d(s[k]) for k in ("x", "b", "w_pre", "w_post", "gate")}
    scale = float(torch.tensor(0.7, dtype=torch.float32))

    def loss(v):
        nb = v["b"]
        if v["w_post"] is not None:
            nb = nb * (nb.square().mean(1, keepdim=True) + EPS).rsqrt() * v["w_post"]
        xo = v["x"] + scale * nb * (1.0 if v["gate"] is None else v["gate"])
        y = xo * (xo.square().mean(1, keepdim=True) + EPS).rsqrt() * v["w_pre"]
        return (dy * y).sum() + (dxo * xo).sum()

    g = torch.Generator().manual_seed(5)
    for name, grad in (("x", "dx"), ("b", "db"), ("w_pre", "dw_pre"), ("w_post", "dw_post"), ("gate", "dgate")):
        if base[name] is None:
            continue
        for _ in range(3):
            v = torch.randn(base[name].shape, generator=g, dtype=torch.float64)
            h = 1e-4
            up, down = dict(base), dict(base)
            up[name], down[name] = base[name] + h * v, base[name] - h * v
            slope = float((loss(up) - loss(down)) / (2 * h))
            gv = d(got[grad]) * v
            tol = (half_step(got[grad].dtype) + 2.0 ** -15) * float(gv.abs().sum()) + 1e-5
            assert abs(float(gv.sum()) - slope) <= tol, (name, float(gv.sum()), slope, tol)


def test_other_stream_and_graph_replays():
    """The calls on a stream of their own, then captured and replayed with eager work in between."""
    s = make(64, 1001, BF16, BF16, "shared", True, seed=21)
    x_out, y = forward(s, 0, 0)
    got = backward(s, x_out)
    side = torch.cuda.Stream()
    xo2, y2 = torch.empty_like(x_out), torch.empty_like(y)
    out = {k: torch.empty_like(v) for k, v in got.items()}
    ws = torch.empty(R.join_workspace_bytes(s["plan"], 64), dtype=torch.uint8, device="cuda")

    def step():
        R.join_forward(s["plan"], s["x"], s["b"], s["w_post"], s["gate"], s["w_pre"], xo2, y2)
        R.join_backward(s["plan"], s["dy"], s["dxo"], xo2, s["b"], s["w_post"], s["gate"], s["w_pre"], out["dx"],
                        out["db"], out["dw_post"], out["dgate"], out["dw_pre"], ws)

    def same():
        torch.cuda.synchronize()
        return torch.equal(xo2, x_out) and torch.equal(y2, y) and all(torch.equal(out[k], got[k]) for k in got)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for v in (xo2, y2, ws, *out.values()):
            v.fill_(1)
        graph.replay()
        assert same()
        (torch.ones(1000, device="cuda") * 2).sum().item()
