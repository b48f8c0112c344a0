"""Helpers of the tests of the operators beside the layer: buffers with odd
strides and guarded padding, and the comparison against 64-bit values."""
import torch

BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
CANARY = -77.0


def half_step(dtype) -> float:
    """Half a rounding step, relative to the value."""
    return torch.finfo(dtype).eps / 2


def strided(rows: int, cols: int, dtype, pad: int = 0, offset: int = 0, device="cuda"):
    """A [rows, cols] view, rows cols + pad elements apart, that starts `offset` elements into its storage,
    which holds the canary everywhere; returns (view, storage)."""
    store = torch.full((rows * (cols + pad) + offset + pad + 8,), CANARY, dtype=dtype, device=device)
    return store[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], store


def fill(view, values):
    view.copy_(values)
    return view


def padding_kept(view, store) -> bool:
    """Whether everything of the storage outside the view still holds the canary."""
    seen = store.clone()
    off = view.storage_offset() - store.storage_offset()
    rows, cols = view.shape
    torch.as_strided(seen, (rows, cols), (view.stride(0), 1), seen.storage_offset() + off).fill_(CANARY)
    return bool((seen == CANARY).all())


def assert_within(got, want, tol, what: str):
    """|got - want| <= tol element by element, all in 64 bits."""
    got, want, tol = got.double().cpu(), want.double().cpu(), tol.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    off = (got - want).abs() - tol
    worst = int(off.argmax())
    assert off.max() <= 0, (f"{what}: {int((off > 0).sum())} of {off.numel()} outside, worst at {worst}: got "
                            f"{got.flatten()[worst]:.9g} want {want.flatten()[worst]:.9g} tol "
                            f"{tol.flatten()[worst]:.3g}")
