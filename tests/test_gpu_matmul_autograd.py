"""moe_grouped_matmul inside torch's graph: gradients of its inputs against float64, and calls that record none."""
import numpy as np
import pytest

import moe_layer_forward_amd as moe

pytestmark = pytest.mark.gpu


def _torch():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def _inputs(dt, gather, past=0, seed=0):
    torch = _torch()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    sizes, N, K = [70, 0, 1, 133, 20], 72, 136
    rows = sum(sizes) + past
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
    x_rows = 40 if gather else rows
    idx = torch.randint(0, x_rows, (rows,), generator=gen, device="cuda", dtype=torch.int32) if gather else None
    if gather:
        idx[:8] = 3  # gathered often
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    x = torch.randn((x_rows, K), generator=gen, device="cuda").to(dtype)
    w = torch.randn((len(sizes), N, K), generator=gen, device="cuda").to(dtype)
    dy = torch.randn((rows, N), generator=gen, device="cuda").to(dtype)
    return off, idx, x, w, dy


def _reference(off, idx, x, w, dy):
    """(dx, dw) in float64, and the same sums of magnitudes."""
    torch = _torch()
    o = off.tolist()
    out = []
    for f in (lambda t: t.double().cpu(), lambda t: t.double().cpu().abs()):
        x6, w6, dy6 = f(x), f(w), f(dy)
        at = torch.arange(len(x)) if idx is None else idx.cpu().long()
        dx, dw = torch.zeros_like(x6), torch.zeros_like(w6)
        for g in range(len(w)):
            r = slice(o[g], o[g + 1])
            dx.index_add_(0, at[r], dy6[r] @ w6[g])
            dw[g] = dy6[r].T @ x6[at[r]]
        out.append((dx, dw))
    return out


@pytest.mark.parametrize("past", [0, 31])
@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gathered"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradients_of_the_inputs(dt, gather, past):
    """Sums of at most `depth` products in fp32, (depth + 16) 2^-23 of their magnitudes, then one rounding to the
    inputs' type, 2^-8 or 2^-23 of the value.  Rows past the last group contribute nothing."""
    torch = _torch()
    off, idx, x, w, dy = _inputs(dt, gather, past)
    if past:
        dy[-past:] = 0.0  # a loss over the rows that exist
    x.requires_grad_(), w.requires_grad_()
    y = moe.moe_grouped_matmul(x, w, off, row_index=idx)
    assert y.requires_grad and y.dtype == x.dtype
    with torch.no_grad():
        plain = moe.moe_grouped_matmul(x, w, off, row_index=idx)
    assert not plain.requires_grad and torch.equal(y[:int(off[-1])], plain[:int(off[-1])])
    y.backward(dy)
    (dx, dw), (ax, aw) = _reference(off, idx, x.detach(), w.detach(), dy)
    depth = dy.shape[0] * w.shape[1]
    out = 2.0 ** -8 if dt == "bf16" else 2.0 ** -23
    for name, got, want, mag in (("dx", x.grad, dx, ax), ("dw", w.grad, dw, aw)):
        assert got.dtype == x.dtype
        err = (got.double().cpu() - want).abs()
        assert bool((err <= out * want.abs() + (depth + 16) * 2.0 ** -23 * mag).all()), name
    # the same bits from a second pass
    first = x.grad.clone(), w.grad.clone()
    x.grad = w.grad = None
    moe.moe_grouped_matmul(x, w, off, row_index=idx).backward(dy)
    assert torch.equal(x.grad, first[0]) and torch.equal(w.grad, first[1])


def test_float32_results_of_bf16_operands():
    torch = _torch()
    off, idx, x, w, dy = _inputs("bf16", False)
    x.requires_grad_(), w.requires_grad_()
    y = moe.moe_grouped_matmul(x, w, off, y_dtype=moe.MOE_F32)
    assert y.dtype == torch.float32
    (y * dy.float()).sum().backward()  # dy is exact in bf16
    assert torch.equal(x.grad, moe.moe_grouped_matmul_dx(dy, w.detach(), off))
    assert torch.equal(w.grad, moe.moe_grouped_matmul_dw(dy, x.detach(), off))


def test_only_the_gradients_that_are_asked_for():
    torch = _torch()
    off, idx, x, w, dy = _inputs("f32", True)
    w.requires_grad_()
    moe.moe_grouped_matmul(x, w, off, row_index=idx).backward(dy)
    assert x.grad is None and w.grad is not None
    w = w.detach()
    x.requires_grad_()
    moe.moe_grouped_matmul(x, w, off, row_index=idx).sum().backward()  # an expanded dy
    assert x.grad is not None and w.grad is None
    # one group without offsets, a row index outside x (moved inside, as the product does)
    x.grad = None
    bad = idx.clone()
    bad[5], bad[6] = -3, 2 ** 31 - 1
    moe.moe_grouped_matmul(x, w[:1].contiguous(), None, row_index=bad).backward(dy)
    assert bool(torch.isfinite(x.grad).all())


def test_calls_without_a_graph():
    torch = _torch()
    off, _, x, w, dy = _inputs("bf16", False)
    out = torch.empty((x.shape[0], w.shape[1]), dtype=x.dtype, device="cuda")
    p = torch.nn.Parameter(w)
    assert moe.moe_grouped_matmul(x, p, off, out=out) is out and not out.requires_grad
    with torch.no_grad():
        y = moe.moe_grouped_matmul(x, p, off)
    assert not y.requires_grad and torch.equal(y, out)
    assert not moe.moe_grouped_matmul(x, w, off).requires_grad
    with pytest.raises(ValueError):
        moe.moe_grouped_matmul(x.float(), p, off)
    with pytest.raises(ValueError):
        moe.moe_grouped_matmul(x, p, None)


def test_no_rows_have_zero_gradients():
    torch = _torch()
    x = torch.empty((0, 16), device="cuda", requires_grad=True)
    w = torch.randn((2, 8, 16), device="cuda", requires_grad=True)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    idx = torch.zeros(0, dtype=torch.int32, device="cuda")
    for i in (None, idx):
        w.grad = None
        moe.moe_grouped_matmul(x, w, off, row_index=i).sum().backward()
        assert bool((w.grad == 0).all()) and x.grad.shape == (0, 16)
