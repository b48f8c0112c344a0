"""Tensors in other shapes than rows and columns, and bits held as integers, give the same bits; what cannot be read on
the device is refused before any launch."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests.block_helpers import BF16, F32

pytestmark = pytest.mark.gpu


def rnd(*shape, dtype=BF16, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def refused(call, text):
    with pytest.raises(R.MoeError) as ei:
        call()
    assert ei.value.code == -1 and text in str(ei.value), str(ei.value)


def test_join_in_other_shapes():
    m, dim = 6, 72
    j = R.Join(dim, BF16, residual=F32)
    x, b, w = rnd(m, dim, dtype=F32), rnd(m, dim, seed=1), rnd(dim, seed=2)
    x_out, y = torch.empty_like(x), torch.empty_like(b)
    R.join_forward(j, x, b, w, None, w, x_out, y)
    for other in (b.view(torch.int16), b.view(m, 8, 9), b.flatten(), b.view(torch.uint8), torch.cat([b, b])):
        x2, y2 = torch.empty(2, 3, dim, dtype=F32, device="cuda"), torch.full((m + 2, dim), 3.0, dtype=BF16, device="cuda")
        R.join_forward(j, x, other, w.view(1, dim), None, w.view(torch.int16), x2, y2)
        assert torch.equal(x2.view(m, dim), x_out) and torch.equal(y2[:m], y) and (y2[m:] == 3).all()
    table = torch.zeros(m, 3, 8, 9, dtype=BF16, device="cuda")
    table[:, 1] = b.view(m, 8, 9)
    y2 = torch.empty_like(y)
    R.join_forward(R.Join(dim, BF16, residual=F32, b_stride=3 * dim), x, table[:, 1], w, None, w, torch.empty_like(x), y2)
    assert torch.equal(y2, y)
    refused(lambda: R.join_forward(j, x, table[:, 1], w, None, w, x_out, y), "its rows do not lie")


def test_grouped_in_other_shapes():
    groups, n, k, rows = 3, 40, 24, 12
    g = R.Grouped(groups, n, k, BF16)
    x, w = rnd(rows, k), rnd(groups, n, k, seed=1)
    off = torch.tensor([0, 5, 5, 12], dtype=torch.int32, device="cuda")
    y = torch.empty(rows, n, dtype=BF16, device="cuda")
    R.grouped_forward(g, x, w, off, y)
    for xo, wo in ((x.view(torch.int16), w.view(groups * n, k)), (x.view(rows, 4, 6), w.flatten()),
                   (torch.cat([x, x])[:rows], w.view(torch.uint8)), (x, w.view(groups, 5, 8, k))):
        y2 = torch.empty(2, rows // 2, n, dtype=BF16, device="cuda")
        R.grouped_forward(g, xo, wo, off.view(1, groups + 1), y2)
        assert torch.equal(y2.view(rows, n), y)
    one = R.Grouped(1, n, k, BF16)
    ends = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    y1, y2 = torch.empty_like(y), torch.empty_like(y)
    R.grouped_forward(one, x, w[1], ends, y1)
    R.grouped_forward(one, x, w[1:2], ends, y2)
    assert torch.equal(y1, y2)
    refused(lambda: R.grouped_forward(g, x, w, off.long(), y), "must be int32")
    refused(lambda: R.grouped_forward(g, x, w, off.cpu(), y), "not on the device")
    refused(lambda: R.grouped_forward(g, x.cpu(), w, off, y), "not on the device")
    refused(lambda: R.grouped_forward(g, x, w, off, y[:-1]), "its rows do not lie")
    refused(lambda: R.grouped_backward_w(g, y, x, off, w.cpu()), "not on the device")


def test_adapters_on_the_host():
    m, n, k, rank = 5, 32, 64, 8
    x, w, a, b = rnd(m, k), rnd(n, k, seed=1), rnd(2, rank, k, seed=2), rnd(2, n, rank, seed=3)
    index = torch.tensor([0, 1, -1, 0, 1], dtype=torch.int32, device="cuda")
    factor = torch.ones(2, device="cuda")
    out, again = (torch.empty(m, n, dtype=BF16, device="cuda") for _ in range(2))
    p = R.Adapters(a, b, factor)
    ws = torch.empty(R.adapter_workspace_bytes(p, m), dtype=torch.uint8, device="cuda")
    R.adapter_project(p, x, w, index, out, ws)
    R.adapter_project(R.Adapters(a, b, factor), x.view(m, 8, 8), w.flatten(), index.view(m, 1), again.view(1, m, n), ws)
    assert torch.equal(out, again)
    for q in (R.Adapters(a.cpu(), b, factor), R.Adapters(a, b.cpu(), factor), R.Adapters(a, b, factor.cpu())):
        refused(lambda: R.adapter_project(q, x, w, index, out, ws), "not on the device")
    refused(lambda: R.adapter_project(p, x, w, index, out, ws.cpu()), "not on the device")
    refused(lambda: R.adapter_project(p, x, w, index.long(), out, ws), "must be int32")


def test_a_copied_description():
    m, n, k, rank = 5, 32, 64, 8
    x, w, a, b = rnd(m, k), rnd(n, k, seed=1), rnd(2, rank, k, seed=2), rnd(2, n, rank, seed=3)
    index = torch.tensor([0, 1, -1, 0, 1], dtype=torch.int32, device="cuda")
    p = R.Adapters(a, b)
    ws = torch.empty(R.adapter_workspace_bytes(p, m), dtype=torch.uint8, device="cuda")
    out, again = (torch.empty(m, n, dtype=BF16, device="cuda") for _ in range(2))
    R.adapter_project(p, x, w, index, out, ws)
    R.adapter_project(R.Adapters.from_buffer_copy(p), x, w, index, again, ws)
    assert torch.equal(out, again)
