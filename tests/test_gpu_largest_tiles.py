"""The largest tiles of the gated and the 4-bit products where other tests reach smaller ones: each size is held against
the library's rule first, so that a test of the largest tiles is one."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests import test_gpu_gated as gated
from tests import test_gpu_mx as mx
from tests.block_helpers import BF16, F32, FP16, padding_kept, strided
from tests.test_gpu_wide_tiles import EDGES, PLAIN_GATED

pytestmark = pytest.mark.gpu


def largest(sizes, columns, terms, before=0, after=0, mx=False):
    """Holds a call of `columns` columns of weights (of both matrices in a gated forward pass) and sums of `terms` terms
    against the rule, which takes the largest tiles from 768 of them on (a row tile has 256 rows, and every group half a
    partial one) where groups have 64 rows or more in the mean and the sums are whole steps."""
    rows, groups = before + sum(sizes) + after, len(sizes)
    row_tiles = -(-rows // 256) if groups == 1 else rows // 256 + min(groups, rows) // 2
    assert row_tiles * -(-columns // 256) >= 768 and rows // groups >= 64
    assert terms % 1024 == 0 if mx else terms % 64 == 0 and terms >= 256


def largest_of(way, sizes, n, k, **more):
    largest(sizes, {"forward": 2 * n, "hidden": n, "input": k}[way], n if way == "input" else k, **more)


WIDTHS = {"forward": (1288, 256), "hidden": (2568, 256), "input": (256, 2568)}   # (n, k): the last tile of columns has 8


def bad_offsets(what, ends, rows):
    bad = list(ends)
    if what == "descending":
        bad[20], bad[40] = bad[40], bad[20]
    elif what == "before":
        bad[0] = -5
    elif what == "behind":
        bad[-1] = rows + 300
    else:
        bad.reverse()
    return torch.tensor(bad, dtype=torch.int32, device="cuda")


BAD = pytest.mark.parametrize("what", ["descending", "before", "behind", "reversed"])


@BAD
@pytest.mark.parametrize("way", gated.WAYS)
def test_bad_offsets_are_reported(way, what):
    n, k = WIDTHS[way]
    largest_of(way, EDGES, n, k, before=3, after=2)
    s = gated.make(EDGES, n, k, BF16, seed=40, pad=8, offset=8, before=3, after=2)
    off, st = bad_offsets(what, s["ends"], s["rows"]), gated.status_word()
    outs = [gated.output(s, k if way == "input" else n, BF16) for _ in range(1 if way == "input" else 3)]
    views = [v for v, _ in outs]
    if way == "forward":
        R.gated_forward(s["plan"], s["x"], s["w_gate"], s["w_up"], off, *views, status=st)
    elif way == "hidden":
        R.gated_backward_h(s["plan"], s["dy"], s["w_down"], s["gate"], s["up"], off, *views, status=st)
    else:
        R.gated_backward_x(s["plan"], s["dgate"], s["dup"], s["w_gate"], s["w_up"], off, *views, status=st)
    torch.cuda.synchronize()
    assert int(st) == R.MOE_STATUS_BAD_OFFSETS and all(padding_kept(*v) for v in outs)


@BAD
@PLAIN_GATED
def test_bad_offsets_are_reported_in_4_bits(of_two, what):
    n = 1288 if of_two else 2568
    largest(EDGES, 2568 + 8 * of_two, 1024, before=3, after=2, mx=True)
    s = mx.make(EDGES, n, 1024, seed=41, pad=16, offset=16, before=3, after=2)
    s["off"] = bad_offsets(what, s["ends"], s["rows"])
    (out, store), st = strided(s["rows"], n, BF16, 16, 16), gated.status_word()
    mx.run(s, of_two, out, st)
    torch.cuda.synchronize()
    assert int(st) == R.MOE_STATUS_BAD_OFFSETS and padding_kept(out, store)


@PLAIN_GATED
def test_nan_stays_in_its_group_in_4_bits(of_two):
    """Blocks of NaN in the rows and the weights of groups that end in the middle of a tile, and of one that has whole ones."""
    n = 1288 if of_two else 2568
    largest(EDGES, 2568 + 8 * of_two, 1024, before=3, after=2, mx=True)
    s = mx.make(EDGES, n, 1024, seed=42, before=3, after=2)
    want = mx.run(s, of_two)
    apart = torch.zeros(s["rows"], dtype=torch.bool, device="cuda")
    for group in (1, 11, 23):   # of 17, 512 and 257 rows
        a, b = s["ends"][group:group + 2]
        apart[a:b] = True
        s["x"][1][a:b] = 255
        for _, scale in (s["w"], s["w2"]):
            scale.view(len(EDGES), n, -1)[group] = 255
    got = mx.run(s, of_two)
    assert want.isfinite().all() and torch.equal(got[~apart], want[~apart]) and got[apart].isnan().all()
    assert (got[:3] == 0).all() and (got[-2:] == 0).all()


@pytest.mark.parametrize("way", gated.WAYS)
def test_weights_past_32_bits(way):
    """Groups whose element offsets pass 2^31 and byte offsets 2^32."""
    sizes, terms, columns = [1500, 2900], 256, 11008
    n, k = {"forward": (columns // 2, terms), "hidden": (columns, terms), "input": (terms, columns)}[way]
    largest_of(way, sizes, n, k)
    s = gated.make(sizes, n, k, BF16, seed=43)
    rows, cols = (k, n) if way == "hidden" else (n, k)
    apart = (1 << 31) + 64
    store = torch.zeros(apart + rows * cols, dtype=BF16, device="cuda")
    far = torch.as_strided(store, (2, rows, cols), (apart, cols, 1))
    dense = s["w_down" if way == "hidden" else "w_gate"].view(2, rows, cols)
    far.copy_(dense)
    over = {"down_group_stride": apart} if way == "hidden" else {"w_group_stride": apart}
    plan = R.Gated(2, n, k, BF16, act=s["act"], limit=s["limit"], **over)
    out = []
    for p, w in ((plan, far), (s["plan"], dense)):
        got = [torch.empty((s["rows"], k if way == "input" else n), dtype=BF16, device="cuda") for _ in range(3)]
        if way == "forward":
            R.gated_forward(p, s["x"], w, w, s["off"], *got)
        elif way == "hidden":
            R.gated_backward_h(p, s["dy"], w, s["gate"], s["up"], s["off"], *got)
        else:
            R.gated_backward_x(p, s["dgate"], s["dup"], w, w, s["off"], got[0])
            got = got[:1]
        out.append(got)
    assert all(torch.equal(a, b) for a, b in zip(*out))


@PLAIN_GATED
def test_weights_past_32_bits_in_4_bits(of_two):
    sizes, columns = [1500, 2900], 11008
    n = columns // 2 if of_two else columns
    largest(sizes, columns, 1024, mx=True)
    s = mx.make(sizes, n, 1024, seed=44)
    want = mx.run(s, of_two)
    apart = (1 << 32) + (1 << 20)
    store = torch.zeros(apart + n * 512, dtype=torch.uint8, device="cuda")
    far = torch.as_strided(store, (2, n, 512), (apart, 512, 1))
    far.copy_(s["w"][0].view(2, n, 512))
    plan = R.Mx(2, n, 1024, BF16, act=s["act"], limit=s["limit"], w_group_stride=apart)
    out = torch.empty_like(want)
    if of_two:   # both halves far: the second matrix as the first one
        want = torch.empty_like(out)
        near = R.Mx(2, n, 1024, BF16, act=s["act"], limit=s["limit"])
        R.mx_gated(near, *s["x"], *s["w"], s["w"][0], s["w2"][1], s["off"], want)
        R.mx_gated(plan, *s["x"], far, s["w"][1], far, s["w2"][1], s["off"], out)
    else:
        R.mx_forward(plan, *s["x"], far, s["w"][1], s["off"], out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("t", [BF16, FP16], ids=["bf16", "fp16"])
def test_odd_number_of_outputs(t):
    """Rows of weights are whole, their number is any: the last outputs one by one, at odd addresses, gate and up beside h."""
    n, k = 1283, 256
    largest_of("forward", EDGES, n, k, before=3, after=2)
    gated.check_forward(gated.make(EDGES, n, k, t, seed=45, pad=8, before=3, after=2))


@PLAIN_GATED
@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
def test_odd_number_of_outputs_in_4_bits(of_two, out):
    n = 1283 if of_two else 2565
    largest(EDGES, 2565 + of_two, 1024, before=3, after=2, mx=True)
    mx.check(mx.make(EDGES, n, 1024, seed=46, before=3, after=2, out=out), of_two)
