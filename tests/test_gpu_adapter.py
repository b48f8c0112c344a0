"""moe_adapter_project against W x + factor B (A x) in 64 bits.

Tolerances. Sums as in the grouped products: a term passes at most 32 additions
inside a matrix instruction, one per 32 terms of its sum, one per slice of
256 or more where the sum over k is cut, and one per term of the short sum over
the rank (three 16-bit terms per value at most), each off by at most 2^-23 of
the sum of the absolute terms. u = factor A x enters the second product in f32
(up to 64 tokens), or as 16-bit terms that leave at most a piece of it: two bf16
terms 2^-16 (half a step of 2^-8 each), two fp16 terms 2^-22 and half the
smallest fp16 step, three bf16 terms 2^-24. Then one rounding of the output."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests.block_helpers import BF16, F32, FP16, assert_within, fill, half_step, padding_kept, strided

pytestmark = pytest.mark.gpu


def make(m, n, k, rank, adapters, t, seed, pad=0, offset=0, order="mixed", scale=1.0):
    g = torch.Generator().manual_seed(seed)
    s = {"m": m, "n": n, "k": k, "rank": rank, "adapters": adapters, "t": t, "pad": pad, "offset": offset}
    s["x"] = fill(strided(m, k, t, pad, offset)[0], torch.randn((m, k), generator=g))
    s["w"] = fill(strided(n, k, t, pad, offset)[0], torch.randn((n, k), generator=g))
    s["a"] = fill(strided(adapters * rank, k, t, pad, offset)[0], scale * torch.randn((adapters * rank, k), generator=g))
    s["b"] = fill(strided(adapters * n, rank, t, pad, offset)[0], torch.randn((adapters * n, rank), generator=g) / scale)
    s["factor"] = (torch.rand(adapters, generator=g) + 0.5).cuda()
    index = torch.randint(-1, adapters, (m,), generator=g)
    if order == "segments":
        index = index.sort().values
    s["index"] = index.to(torch.int32).cuda()
    return s


def plan(s, out, factor=True):
    r, k, n, pad = s["rank"], s["k"], s["n"], s["pad"]
    a = torch.as_strided(s["a"], (s["adapters"], r, k), (r * (k + pad), k + pad, 1), s["a"].storage_offset())
    b = torch.as_strided(s["b"], (s["adapters"], n, r), (n * (r + pad), r + pad, 1), s["b"].storage_offset())
    return R.Adapters(a, b, s["factor"] if factor else None, out=out, x_stride=k + pad, w_stride=k + pad,
                      out_stride=n + pad)


def want(s, out, factor=True):
    m, n, k, r = s["m"], s["n"], s["k"], s["rank"]
    x, w = s["x"].double(), s["w"].double()
    a, b = s["a"].double().reshape(-1, r, k), s["b"].double().reshape(-1, n, r)
    v, mag, left = x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous(), torch.zeros((m, n), dtype=torch.float64, device="cuda")
    for i in range(s["adapters"]):
        rows = (s["index"] == i).nonzero()[:, 0]
        if not rows.numel():
            continue
        f = float(s["factor"][i]) if factor else 1.0
        at, bt = a[i].t().contiguous(), b[i].t().contiguous()
        u = f * (x[rows] @ at)
        v[rows] += u @ bt
        mag[rows] += f * (x[rows].abs() @ at.abs()) @ bt.abs()
        if m <= 64:
            piece, least = 0.0, 0.0
        elif s["t"] == FP16:
            piece, least = 2.0 ** -22, 2.0 ** -25
        else:
            piece, least = 2.0 ** -24 if out == F32 else 2.0 ** -16, 0.0
        left[rows] += (piece * u.abs() + least) @ bt.abs()
    steps = k / 32 + k / 256 + 3 * r + 40
    tol = half_step(out) * v.abs() + steps * 2.0 ** -23 * mag + left + 1e-30 + (2.0 ** -25 if out == FP16 else 0.0)
    return v, tol


def workspace(p, m):
    n = R.adapter_workspace_bytes(p, m)
    assert n > 0
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN wherever it is read before it is written


def run(s, out, factor=True, status=None):
    p = plan(s, out, factor)
    y, store = strided(s["m"], s["n"], out, s["pad"], s["offset"])
    R.adapter_project(p, s["x"], s["w"], s["index"], y, workspace(p, s["m"]), status)
    torch.cuda.synchronize()
    assert padding_kept(y, store)
    return y


def check(s, out, factor=True):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = run(s, out, factor, status)
    assert int(status) == 0
    v, tol = want(s, out, factor)
    assert_within(y, v, tol, f"m {s['m']} n {s['n']} k {s['k']} rank {s['rank']} x{s['adapters']} {s['t']}->{out}")
    return y


TOKENS = [1, 2, 15, 16, 17, 33, 64, 65, 130, 600]


@pytest.mark.parametrize("m", TOKENS)
@pytest.mark.parametrize("t", [BF16, FP16], ids=["bf16", "fp16"])
def test_tokens(m, t):
    check(make(m, 192, 320, 16, 5, t, seed=m), t)
    check(make(m, 72, 1000, 40, 3, t, seed=m, pad=8, offset=8, order="segments"), F32)
    check(make(m, 257, 515, 7, 4, t, seed=m, pad=1, offset=3), F32)
    check(make(m, 65, 67, 70, 2, t, seed=m, order="segments"), t, factor=False)


@pytest.mark.parametrize("m", [3, 64, 90, 520])
@pytest.mark.parametrize("rank", [1, 3, 8, 17, 32, 33, 64, 65, 200])
def test_ranks(m, rank):
    check(make(m, 136, 264, rank, 6, BF16, seed=rank), F32)
    check(make(m, 40, 96, rank, 2, FP16, seed=rank), FP16)


@pytest.mark.parametrize("m", [5, 64, 300])
@pytest.mark.parametrize("n,k", [(1, 1), (1, 64), (64, 1), (7, 4096), (4096, 7), (64, 64), (200, 2048)])
def test_widths(m, n, k):
    check(make(m, n, k, 16, 3, BF16, seed=1), BF16)


@pytest.mark.parametrize("m", [8, 64, 100, 1200])
def test_adapters(m):
    for adapters in (1, 2, 70, 1024):
        check(make(m, 64, 128, 8, adapters, BF16, seed=adapters), BF16)
    for order in ([-1] * m, [0] * m, [2] * m, [0, 2] * (m // 2)):
        s = make(m, 64, 128, 8, 3, FP16, seed=5)
        s["index"] = torch.tensor(order, dtype=torch.int32, device="cuda")
        check(s, F32)


@pytest.mark.parametrize("m", [40, 100, 700])
def test_token_does_not_depend_on_its_neighbours(m):
    """A token alone among the others' adapters gives the same bits wherever it stands; the same call gives the same bits."""
    s = make(m, 136, 264, 16, 5, BF16, seed=4)
    y = run(s, F32)
    assert torch.equal(y, run(s, F32))
    perm = torch.randperm(m, generator=torch.Generator().manual_seed(1)).cuda()
    s2 = dict(s)
    s2["x"], s2["index"] = s["x"][perm].contiguous(), s["index"][perm].contiguous()
    assert torch.equal(run(s2, F32), y[perm])


@pytest.mark.parametrize("m", [40, 100, 700])
def test_infinities_stay_with_their_tokens(m):
    s = make(m, 136, 264, 16, 5, BF16, seed=4)
    s["index"][:5] = torch.arange(5, dtype=torch.int32)
    clean = run(s, BF16)
    r, n = s["rank"], s["n"]
    s["a"][r:2 * r] = float("nan")
    s["b"][3 * n:4 * n] = float("inf")
    hurt = (s["index"] == 1) | (s["index"] == 3)
    y = run(s, BF16)
    assert y[s["index"] == 1].isnan().all() and not torch.isfinite(y[s["index"] == 3]).any()
    assert torch.equal(y[~hurt], clean[~hurt])
    s["x"][7] = float("inf")
    keep = ~hurt
    keep[7] = False
    assert torch.equal(run(s, BF16)[keep], clean[keep])


@pytest.mark.parametrize("m", [30, 100, 600])
def test_low_rank_values_past_the_range_of_fp16(m):
    """A x up to 2^18, against B of the size that brings the product back to order one."""
    s = make(m, 72, 264, 40, 3, FP16, seed=2, scale=2.0 ** 10)
    s["x"] *= 8
    assert float((s["x"].double() @ s["a"][:40].double().t().contiguous()).abs().max()) > 2.0 ** 17
    check(s, F32)


@pytest.mark.parametrize("m", [20, 100])
def test_bad_index_is_reported(m):
    s = make(m, 72, 64, 8, 3, BF16, seed=3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["index"][4], s["index"][9], s["index"][11] = 3, -2, 2 ** 31 - 1
    y = run(s, F32, status=status)
    assert int(status) == R.MOE_STATUS_BAD_ADAPTER
    s["index"][4], s["index"][9], s["index"][11] = -1, -1, -1
    assert torch.equal(y, check(s, F32))


def test_positions_past_32_bits():
    n, k, rank, m = 64, 128, 16, 600
    stride = R.MOE_GROUPED_MAX_STRIDE
    s = make(m, n, k, rank, 3, BF16, seed=8)
    big = torch.zeros((m - 1) * stride + k, dtype=BF16, device="cuda")
    view = torch.as_strided(big, (m, k), (stride, 1))
    view.copy_(s["x"])
    for count in (40, m):
        apart = 2 ** 30 + 64
        far = torch.zeros(2 * apart + rank * k, dtype=BF16, device="cuda")
        a = torch.as_strided(far, (3, rank, k), (apart, k, 1))
        a.copy_(s["a"].view(3, rank, k))
        p = R.Adapters(a, s["b"].view(3, n, rank), s["factor"], out=F32, x_stride=stride)
        y = torch.empty((count, n), dtype=F32, device="cuda")
        R.adapter_project(p, view[:count], s["w"], s["index"][:count], y, workspace(p, count))
        part = {**s, "m": count, "x": s["x"][:count], "index": s["index"][:count]}
        v, tol = want(part, F32)
        assert_within(y, v, tol, f"m {count}")
        del far, a


def test_one_workspace_serves_fewer_tokens():
    s = make(300, 72, 64, 8, 3, BF16, seed=3)
    p = plan(s, F32)
    ws = workspace(p, 300)
    full = run(s, F32)
    for m in (300, 1, 64, 65, 7):
        y = torch.empty((m, 72), dtype=F32, device="cuda")
        R.adapter_project(p, s["x"][:m], s["w"], s["index"][:m], y, ws)
        v, tol = want({**s, "m": m, "x": s["x"][:m], "index": s["index"][:m]}, F32)
        assert_within(y, v, tol, f"m {m}")
    assert torch.equal(run(s, F32), full)


@pytest.mark.parametrize("m", [5, 200])
def test_other_stream_and_graph_replays(m):
    s = make(m, 136, 264, 16, 5, BF16, seed=4)
    p = plan(s, BF16)
    y = run(s, BF16)
    again, ws = torch.empty_like(y), workspace(p, m)

    def step():
        R.adapter_project(p, s["x"], s["w"], s["index"], again, ws)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert torch.equal(again, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        again.fill_(1)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, y)
        (torch.ones(1000, device="cuda") * 2).sum().item()
    s["index"].copy_(s["index"].flip(0))
    graph.replay()
    v, tol = want(s, BF16)
    assert_within(again, v, tol, "after new indices")
