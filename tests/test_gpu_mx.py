"""moe_mx_* against the format and the products in 64 bits.

Tolerances. The rows' codes, scales and f32 values are exact; other types round
the value once. Products of 4-bit elements and powers of two are exact in f32. A
matrix instruction sums 128 of them and adds them to the running sum: a term
passes at most 128 + r / 128 + 1 additions for r terms, each off by at most 2^-23
of the sum of the absolute terms, then one rounding to the output's type (half a
step). The gated product takes the activation's errors of gated_helpers on top."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests.block_helpers import BF16, F32, FP16, assert_within, half_step, padding_kept, strided
from tests.gated_helpers import ACT, STEEPEST, activation, limited
from tests.mx_helpers import quantised, values
from tests.test_gpu_grouped import FEW, MANY, SOME, bounds

pytestmark = pytest.mark.gpu
U8 = torch.uint8
RULES = pytest.mark.parametrize("rule", ["floor", "ceil"])
TYPES = pytest.mark.parametrize("t", [BF16, FP16, F32], ids=["bf16", "fp16", "f32"])


def byte_rows(rows, cols, pad=0, offset=0):
    """A guarded view of byte rows (the canary is 179)."""
    store = torch.full((rows * (cols + pad) + offset + pad + 8,), 179, dtype=U8, device="cuda")
    return store[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], store


def bytes_kept(view, store):
    seen = store.clone()
    torch.as_strided(seen, view.shape, (view.stride(0), 1), view.storage_offset()).fill_(179)
    return bool((seen == 179).all())


def check_rows(x, rule, pad=0, offset=0, out=None):
    """Quantises and dequantises x, compares both, and returns codes and scales."""
    rows, k = x.shape
    out = out or x.dtype
    xv, _ = strided(rows, k, x.dtype, pad, offset)
    xv.copy_(x)
    (codes, cs), (scales, ss) = byte_rows(rows, (k + 1) // 2, pad, offset), byte_rows(rows, (k + 31) // 32, pad, offset)
    p = R.MxRows(k, x.dtype, scale=rule, x_stride=k + pad, code_stride=codes.stride(0), scale_stride=scales.stride(0))
    R.mx_quantise(p, xv, codes, scales)
    want_codes, want_scales = quantised(x.cpu(), rule)
    assert torch.equal(scales.cpu(), want_scales)
    assert torch.equal(codes.cpu(), want_codes)
    assert bytes_kept(codes, cs) and bytes_kept(scales, ss)
    back, store = strided(rows, k, out, pad, offset)
    R.mx_dequantise(R.MxRows(k, out, x_stride=k + pad, code_stride=codes.stride(0), scale_stride=scales.stride(0)), codes,
                    scales, back)
    want = values(codes, scales, k).to(out)   # (one rounding: the 64-bit values have at most 2 bits)
    assert torch.equal(torch.nan_to_num(back, nan=-3.0), torch.nan_to_num(want, nan=-3.0))
    assert padding_kept(back, store)
    return codes, scales


@RULES
@TYPES
@pytest.mark.parametrize("k", [1, 2, 7, 31, 32, 33, 63, 64, 100, 257, 515, 1024, 4097])
def test_rows(k, t, rule):
    gen = torch.Generator().manual_seed(k)
    for i, rows in enumerate((1, 3, 130)):
        x = (torch.randn((rows, k), generator=gen) * torch.exp2(torch.randint(-12, 9, (rows, 1), generator=gen))).to(t).cuda()
        check_rows(x, rule, pad=(0, 1, 8)[i], offset=(0, 3, 16)[i], out=(None, F32, BF16)[i])


@RULES
@pytest.mark.parametrize("t", [BF16, FP16], ids=["bf16", "fp16"])
def test_every_value(t, rule):
    """Every 16-bit pattern, alone in its block, beside a larger one, and among neighbours (infinities and NaN among them)."""
    every = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(t)
    alone = torch.zeros((65536, 32), dtype=t)
    alone[:, 5] = every
    check_rows(alone.cuda(), rule)
    alone[:, 9] = (every.float().abs() * 3.3).to(t)
    check_rows(alone.cuda(), rule)
    check_rows(every.view(2048, 32).cuda(), rule)


@RULES
def test_borders_in_f32(rule):
    """Values at, just below and just above every border between steps and scales, over all exponents."""
    edges = torch.tensor([0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0], dtype=F32)
    edges = torch.cat([edges, torch.nextafter(edges, torch.tensor(0.0)), torch.nextafter(edges, torch.tensor(99.0))])
    rows = []
    for e in list(range(-127, 126, 7)) + [-126, -125, -124, 123, 124, 125]:
        for top in (4.0, 5.9, 6.0, 6.1, 7.9):
            row = torch.zeros(64, dtype=F32)
            row[:45] = torch.ldexp(edges, torch.tensor(e))
            row[45] = row[10] = torch.ldexp(torch.tensor(top), torch.tensor(e))
            row[0::2] *= -1
            rows.append(row)
    x = torch.stack(rows)
    check_rows(torch.where(x.isfinite(), x, 0.0).cuda(), rule)


def test_smallest_and_largest():
    """Subnormal blocks, where the scale stays at 2^-127, blocks of zeros and of negative zeros, and the largest values."""
    tiny = torch.tensor([2.0 ** -149, 2.0 ** -130, 2.0 ** -128, 2.0 ** -127, 1.5 * 2.0 ** -127, 2.0 ** -126, -2.0 ** -126 * 1.99,
                         -0.0], dtype=F32).repeat(4)
    big = torch.full((32,), torch.finfo(F32).max)
    x = torch.stack([tiny, tiny / 2, torch.zeros(32), -torch.zeros(32), big, -big, big / 3])
    for rule in ("floor", "ceil"):
        check_rows(x.cuda(), rule)


def test_scales_outside_a_type():
    """Values past fp16's range become infinite and those below it 0 or subnormal; f32 holds all of them but 4 and 6 times 2^127."""
    codes = torch.arange(256, dtype=torch.int32).to(U8).repeat(256, 1).view(256, 256)[:, :16].contiguous().cuda()
    codes = (codes + 16 * torch.arange(16, device="cuda").to(U8))
    scales = torch.arange(256, dtype=torch.int32).to(U8).view(256, 1).cuda()
    for t in (BF16, FP16, F32):
        x = torch.empty((256, 32), dtype=t, device="cuda")
        R.mx_dequantise(R.MxRows(32, t), codes, scales, x)
        want = values(codes, scales, 32).to(F32).to(t)
        assert torch.equal(torch.nan_to_num(x, nan=-3.0, posinf=1e4, neginf=-1e4),
                           torch.nan_to_num(want, nan=-3.0, posinf=1e4, neginf=-1e4)), t
        assert x[255].isnan().all()


def test_torch_types_and_shapes_of_bytes():
    x = torch.randn((6, 128), generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    codes, scales = check_rows(x, "floor")
    c2 = torch.empty((6, 64), dtype=torch.float4_e2m1fn_x2, device="cuda")
    s2 = torch.empty((6, 4), dtype=torch.float8_e8m0fnu, device="cuda")
    R.mx_quantise(R.MxRows(128, BF16), x.view(2, 3, 128).view(6, 128), c2, s2)
    assert torch.equal(c2.view(U8), codes) and torch.equal(s2.view(U8), scales)


def test_many_rows_and_rows_past_32_bits():
    """More chunks than a workgroup's, rows of one element, and strides that pass 2^31 elements."""
    gen = torch.Generator().manual_seed(3)
    check_rows(torch.randn((70001, 1), generator=gen).cuda(), "floor")
    check_rows(torch.randn((1, 300001), generator=gen).to(BF16).cuda(), "ceil")
    x = torch.randn((3, 64), generator=gen).to(BF16)
    apart = (1 << 30) + 24
    big = torch.zeros(2 * apart + 64, dtype=BF16, device="cuda")
    view = torch.as_strided(big, (3, 64), (apart, 1))
    view.copy_(x)
    codes, scales = torch.empty((3, 32), dtype=U8, device="cuda"), torch.empty((3, 2), dtype=U8, device="cuda")
    R.mx_quantise(R.MxRows(64, BF16, x_stride=apart), view, codes, scales)
    want = quantised(x, "floor")
    assert torch.equal(codes.cpu(), want[0]) and torch.equal(scales.cpu(), want[1])
    R.mx_dequantise(R.MxRows(64, BF16, x_stride=apart), codes, scales, view)
    assert torch.equal(view.cpu().double(), values(*want, 64))


# ---- products -------------------------------------------------------------------------------------
def operand(gen, rows, k, pad, offset, spread):
    """Random codes with scales of a few powers of two, guarded rows; the scales' rows pad a multiple of 4 where codes' are of 16."""
    codes, _ = byte_rows(rows, (k + 1) // 2, pad, offset)
    scales, _ = byte_rows(rows, (k + 31) // 32, pad // 4 * 4 if pad % 16 == 0 else pad, offset)
    codes.copy_(torch.randint(0, 256, codes.shape, generator=gen, dtype=torch.int32).to(U8))
    scales.copy_(torch.randint(127 - spread, 128 + spread, scales.shape, generator=gen, dtype=torch.int32).to(U8))
    return codes, scales


def make(sizes, n, k, seed=0, pad=0, offset=0, before=0, after=0, out=BF16, act="silu", limit=0.0, spread=2, shift=None):
    gen = torch.Generator().manual_seed(seed)
    rows, groups = before + sum(sizes) + after, len(sizes)
    s = {"ends": bounds(sizes, before), "rows": rows, "groups": groups, "n": n, "k": k, "out": out, "pad": pad,
         "offset": offset, "act": act, "limit": limit}
    s["off"] = torch.tensor(s["ends"], dtype=torch.int32, device="cuda")
    s["x"] = operand(gen, rows, k, pad, offset, spread)
    s["w"], s["w2"] = (operand(gen, groups * n, k, pad, offset, spread) for _ in range(2))
    for _, scale in (s["w"], s["w2"]):   # products of about 1
        scale -= 3 + (k.bit_length() // 2 if shift is None else shift)
    s["plan"] = plan(s)
    return s


def plan(s):
    (x, xs), (w, ws) = s["x"], s["w"]
    return R.Mx(s["groups"], s["n"], s["k"], s["out"], act=s["act"], limit=s["limit"], x_stride=x.stride(0),
                x_scale_stride=xs.stride(0), y_stride=s["n"] + s["pad"], w_stride=w.stride(0), w_scale_stride=ws.stride(0))


def sums(s, w):
    x, w = values(*s["x"], s["k"]), values(*w, s["k"]).view(s["groups"], s["n"], s["k"])
    v, mag = (torch.zeros((s["rows"], s["n"]), dtype=torch.float64, device="cuda") for _ in range(2))
    for g, (a, b) in enumerate(zip(s["ends"], s["ends"][1:])):
        if a < b:
            v[a:b], mag[a:b] = x[a:b] @ w[g].t().contiguous(), x[a:b].abs() @ w[g].abs().t().contiguous()
    return v, (129 + s["k"] / 128) * 2.0 ** -23 * mag


def run(s, gated, out=None, st=None, stream=None):
    if out is None:
        out = strided(s["rows"], s["n"], s["out"], s["pad"], s["offset"])[0]
    if gated:
        R.mx_gated(s["plan"], *s["x"], *s["w"], *s["w2"], s["off"], out, st, stream)
    else:
        R.mx_forward(s["plan"], *s["x"], *s["w"], s["off"], out, st, stream)
    return out


def rounded(v, t):
    return half_step(t) * v.abs() + (2.0 ** -25 if t == FP16 else 2.0 ** -130)


def check(s, gated=False):
    out, store = strided(s["rows"], s["n"], s["out"], s["pad"], s["offset"])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    run(s, gated, out, st)
    torch.cuda.synchronize()
    assert int(st) == 0 and padding_kept(out, store)
    what = f"{s['out']} {s['n']}x{s['k']} {s['ends']}"
    v, e = sums(s, s["w"])
    if gated:
        u, eu = sums(s, s["w2"])
        gc, uc = limited(v, u, s["limit"])
        a = activation(gc, s["act"])[0]
        off = STEEPEST * e + ACT * (gc.abs() + e)
        v, e = a * uc, 1.01 * (off * (uc.abs() + eu) + a.abs() * eu) + 2.0 ** -22 * (a * uc).abs()
    assert_within(out, v, rounded(v, s["out"]) + e, what)
    return out


GATED = pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])


@GATED
@pytest.mark.parametrize("n,k", [(64, 256), (128, 512), (136, 288), (8, 1024), (264, 1280), (192, 4096), (16, 32), (65, 768)])
def test_aligned(n, k, gated):
    for i, sizes in enumerate((FEW, SOME, MANY)):
        check(make(sizes, n, k, seed=i, pad=16 * i, offset=16 * i, before=i, after=2 * i, out=(BF16, F32, FP16)[i],
                   act=("silu", "gelu")[i % 2], limit=(0.0, 1.0, 0.5)[i]), gated)


@GATED
@pytest.mark.parametrize("n,k", [(1, 1), (1, 64), (64, 1), (7, 200), (257, 515), (129, 127), (65, 31), (33, 4099), (16, 33)])
def test_any_width_and_alignment(n, k, gated):
    for i, sizes in enumerate((FEW, SOME, MANY)):
        check(make(sizes, n, k, seed=i, before=5 * i, after=i, out=(F32, BF16, FP16)[i]), gated)
    check(make(SOME, n, k, seed=9, pad=3, offset=1, out=F32), gated)
    check(make(FEW, n, k, seed=9, pad=16, offset=5, limit=1.5), gated)


@GATED
@pytest.mark.parametrize("sizes", [[1], [0], [0, 0, 7], [300], [64] * 16, [1] * 700, [0] * 500 + [3] + [0] * 523,
                                   [2, 0] * 512, [4000], [4000, 1]], ids=lambda v: f"{len(v)}x{sum(v)}")
def test_groups(sizes, gated):
    check(make(sizes, 64, 256, seed=2, before=1, after=3), gated)
    if sum(sizes):
        check(make(sizes, 40, 72, seed=3, out=F32), gated)


@GATED
@pytest.mark.parametrize("sizes,n,k", [([700, 0, 900, 450], 1024, 1056), ([2100, 1900, 1, 2100], 2048, 4096), ([3000], 2056, 1024),
                                       ([2100, 1900, 1, 2100], 2048, 4224)], ids=["4 groups", "large tiles", "one group", "tail"])
def test_large_tiles(sizes, n, k, gated):
    check(make(sizes, n, k, seed=4, before=2, after=1), gated)


@pytest.mark.parametrize("k", [512, 515, 800])
def test_odd_elements_past_the_row(k):
    """Whatever lies in the half byte past an odd row, and past the rows, stays out of the sums."""
    s = make(SOME, 40, k, seed=5, pad=16, out=F32)
    first = run(s, False)
    for codes, _ in (s["x"], s["w"]):
        if k % 2:
            codes[:, -1] ^= 0xf0
        torch.as_strided(codes, (codes.shape[0] - 1, 16), (codes.stride(0), 1), codes.storage_offset() + codes.shape[1]).fill_(0x77)
    assert torch.equal(run(s, False), first)


@GATED
def test_scales_at_their_ends(gated):
    """Scales of 0 and 254 in one row meet in products that f32 holds; 255 makes what it enters NaN, and nothing else."""
    s = make([5, 20, 33], 72, 768, seed=6, out=F32, shift=-3, limit=7.0)
    x, w = s["x"][1], s["w"][1]
    x[:, 3], w[:, 3] = 0, 254
    x[:, 7], w[:, 7] = 254, 0
    s["w2"][1][:, 3], s["w2"][1][:, 7] = 254, 0
    check(s, gated)
    clean = run(s, gated)
    x[7, 11] = 255          # row 7 (of the second group)
    w[72 + 4, 20] = 255     # output 4 of the second group
    out = run(s, gated)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[7] = True
    bad[5:25, 4] = True
    assert out[bad].isnan().all() and torch.equal(out[~bad], clean[~bad])


@GATED
def test_captured_and_replayed(gated):
    s = make(MANY, 136, 768, seed=7)
    x = torch.randn((s["rows"], 768), generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    rows = R.MxRows(768, BF16, code_stride=s["x"][0].stride(0), scale_stride=s["x"][1].stride(0))
    out = run(s, gated)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.mx_quantise(rows, x, *s["x"])
        run(s, gated, out)
    for i in range(4):
        x.mul_(-0.7)
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        kept = [v.clone() for v in s["x"]]
        R.mx_quantise(rows, x, *s["x"])
        assert all(torch.equal(a, b) for a, b in zip(kept, s["x"]))
        assert torch.equal(run(s, gated), out), i


def test_two_streams_at_once():
    a, b = make(MANY, 136, 768, seed=8), make(SOME, 200, 512, seed=9)
    want = [run(v, True) for v in (a, b)]
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [torch.empty_like(v) for v in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for v, out, stream in zip((a, b), got, streams):
            run(v, True, out, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@GATED
@pytest.mark.parametrize("ends", [[0, 5, 3, 9], [0, 4, 9, 13], [-2, 4, 6, 9], [9, 6, 3, 0], [1 << 30, 0, (1 << 31) - 1, 2]])
def test_bad_offsets_are_reported(ends, gated):
    s = make([3, 3, 3], 40, 288, seed=10, pad=16)
    s["off"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    out, store = strided(s["rows"], s["n"], BF16, 16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    run(s, gated, out, st)
    torch.cuda.synchronize()
    assert int(st) == R.MOE_STATUS_BAD_OFFSETS and padding_kept(out, store)


@GATED
def test_no_rows(gated):
    s = make([3, 2], 40, 288, seed=11)
    s["x"] = tuple(v[:0] for v in s["x"])
    out = torch.empty((0, 40), dtype=BF16, device="cuda")
    for ends, code in (([0, 0, 0], 0), ([0, 1, 2], R.MOE_STATUS_BAD_OFFSETS)):
        s["off"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        run(s, gated, out, st)
        torch.cuda.synchronize()
        assert int(st) == code


def test_weights_past_32_bits():
    """Groups of codes whose byte offsets pass 2^32."""
    s = make([9, 1, 20], 64, 512, seed=12, out=F32)
    apart = (1 << 31) + (1 << 20)
    big = torch.zeros(2 * apart + 64 * 256, dtype=U8, device="cuda")
    view = torch.as_strided(big, (3, 64, 256), (apart, 256, 1))
    view.copy_(s["w"][0].view(3, 64, 256))
    out = torch.empty((s["rows"], 64), dtype=F32, device="cuda")
    R.mx_forward(R.Mx(3, 64, 512, F32, w_group_stride=apart), *s["x"], view, s["w"][1], s["off"], out)
    assert torch.equal(out, run(s, False))


def test_trained_weights_served_in_4_bits():
    """Experts of the 16-bit gated block quantised, then served: rows to 4 bits, gated product, rows to 4 bits, down
    product. Each step against 64 bits of what the step before gave."""
    gen = torch.Generator().manual_seed(13)
    sizes, n, k, t = [3, 0, 40, 90], 192, 320, BF16
    groups, rows, ends = len(sizes), sum(sizes), bounds(sizes)
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    x = torch.randn((rows, k), generator=gen).to(t).cuda()
    w = {key: (torch.randn((groups, *shape), generator=gen) * 0.08).to(t).cuda()
         for key, shape in (("gate", (n, k)), ("up", (n, k)), ("down", (k, n)))}

    def rows_of(v):
        v = v.reshape(-1, v.shape[-1])
        return check_rows(v, "ceil")

    q = {key: [v.view(groups, -1, v.shape[1]) for v in rows_of(m)] for key, m in w.items()}
    qx = rows_of(x)
    s = {"x": qx, "w": [v.flatten(0, 1) for v in q["gate"]], "w2": [v.flatten(0, 1) for v in q["up"]], "off": off, "ends": ends,
         "rows": rows, "groups": groups, "n": n, "k": k, "out": t, "pad": 0, "offset": 0, "act": "silu", "limit": 7.0}
    s["plan"] = plan(s)
    h = check(s, gated=True)
    s = {**s, "x": rows_of(h), "w": [v.flatten(0, 1) for v in q["down"]], "n": k, "k": n}
    s["plan"] = plan(s)
    y = check(s)
    # and near the 16-bit block: an element in 4 bits is off by at most a sixth of its block's largest (half a step of 2
    # below 6 times the scale), a uniform error of that width over sqrt(3) in the mean, in two operands of two products
    h16 = torch.empty((rows, n), dtype=t, device="cuda")
    R.gated_forward(R.Gated(groups, n, k, t, limit=7.0), x, w["gate"], w["up"], off, h16)
    y16 = torch.empty((rows, k), dtype=t, device="cuda")
    R.grouped_forward(R.Grouped(groups, k, n, t), h16, w["down"], off, y16)
    assert float((y.double() - y16.double()).norm() / y16.double().norm()) < 0.5
