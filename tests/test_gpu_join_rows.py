"""Block joins' gradients where a workgroup takes several rows one after another, at every width class: the sums it
carries from row to row, and gradients written in place. Values and tolerances are those of the tests of the joins."""
import pytest
import torch

import routing_quant_expert_amd as R
from tests import test_gpu_join as join
from tests.block_helpers import BF16, F32, FP16, strided

pytestmark = pytest.mark.gpu

ROWS = 600   # at most 256 workgroups for wide rows: two or three rows each


@pytest.mark.parametrize("dim", [2048, 2050, 5000, 5001, 8192, 8200, 16383, 16384])
@pytest.mark.parametrize("t,res,gate", [(BF16, F32, "shared"), (FP16, FP16, "rows")], ids=["bf16-f32", "fp16-gate-rows"])
def test_several_rows_a_workgroup(dim, t, res, gate):
    s = join.make(ROWS, dim, t, res, gate, True, seed=dim)
    x_out, _ = join.forward(s, 0, 0)
    want, mag = join.formulas(s, x_out)
    join.check_backward(s, join.backward(s, x_out), want, mag)


@pytest.mark.parametrize("dim", [8192, 16384])
@pytest.mark.parametrize("t,res,gate", [(FP16, F32, "rows"), (BF16, BF16, "shared")], ids=["fp16-f32-gate-rows", "bf16"])
def test_several_wide_rows_of_the_other_types(dim, t, res, gate):
    s = join.make(ROWS, dim, t, res, gate, True, seed=dim + 1)
    x_out, _ = join.forward(s, 0, 0)
    want, mag = join.formulas(s, x_out)
    join.check_backward(s, join.backward(s, x_out), want, mag)


@pytest.mark.parametrize("dim", [7, 511, 1001, 2050, 4099, 8192, 8200, 16383, 16384])
@pytest.mark.parametrize("pad,offset", [(0, 0), (5, 3)])
def test_gradients_in_place(dim, pad, offset):
    """dx over dx_out and db over b: the bits of the call with buffers of its own, nothing written beside the rows."""
    s = join.make(ROWS, dim, BF16, F32, "shared", True, seed=dim, pad=pad, offset=offset)
    x_out, _ = join.forward(s, pad, offset)
    got = join.backward(s, x_out, pad, offset)
    dx, dx_store = strided(ROWS, dim, F32, pad, offset)
    db, db_store = strided(ROWS, dim, BF16, pad, offset)
    dx.copy_(s["dxo"])
    db.copy_(s["b"])
    ws = torch.empty(R.join_workspace_bytes(s["plan"], ROWS), dtype=torch.uint8, device="cuda")
    vecs = {k: torch.empty(dim, dtype=F32, device="cuda") for k in ("dw_post", "dgate", "dw_pre")}
    R.join_backward(s["plan"], s["dy"], dx, x_out, db, s["w_post"], s["gate"], s["w_pre"], dx, db, vecs["dw_post"],
                    vecs["dgate"], vecs["dw_pre"], ws)
    torch.cuda.synchronize()
    assert torch.equal(dx, got["dx"]) and torch.equal(db, got["db"])
    assert all(torch.equal(v, got[k]) for k, v in vecs.items())
    assert join.padding_kept(dx, dx_store) and join.padding_kept(db, db_store)
