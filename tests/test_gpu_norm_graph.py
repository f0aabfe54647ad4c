"""The norm as a node of torch's graph and its gradients' types, against float64."""
import pytest

import moe_layer_forward_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _torch():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def _randn(shape, dtype, seed, scale=1.0):
    torch = _torch()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(getattr(torch, dtype))


def _check(dx, dw, dy, h, w, dh, eps=1e-6):
    """dx: two sums of 64 roundings each and a handful of products, 160 u of the magnitudes, and one rounding to its type.
    dw: 40 u a term, a chain of at most rows / 128 terms in a work-group and 150 after it, and one rounding."""
    torch = _torch()
    dy, hd, wd = dy.double(), h.double(), torch.ones(h.shape[1], device="cuda").double() if w is None else w.double()
    m = 1 / ((hd * hd).mean(dim=1, keepdim=True) + eps).sqrt()
    g, n = dy * wd, h.shape[1]
    ref = m * (g - hd * m ** 2 * (g * hd).sum(dim=1, keepdim=True) / n)
    mag = m * (g.abs() + hd.abs() * m ** 2 * (g * hd).abs().sum(dim=1, keepdim=True) / n)
    if dh is not None:
        ref, mag = ref + dh.double(), mag + dh.double().abs()
    err, bound = (dx.double() - ref).abs(), 160 * U * mag + torch.finfo(dx.dtype).eps / 2 * ref.abs() + 2.0 ** -126
    assert bool((err <= bound).all()), float((err / bound).max())
    if dw is not None:
        ref, mag = (dy * hd * m).sum(dim=0), (dy * hd * m).abs().sum(dim=0)
        err = (dw.double() - ref).abs()
        bound = (190 + len(h) / 128) * U * mag + torch.finfo(dw.dtype).eps / 2 * ref.abs() + 2.0 ** -126
        assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("rows,cols", [(1, 7), (33, 200), (4, 2049), (900, 72), (2100, 511), (700, 2048), (40, 7168), (300, 8193),
                                       (3, 16392), (5300, 7168)])
@pytest.mark.parametrize("wdt", ["float32", "bfloat16", None])
def test_an_fp32_gradient_of_bf16_rows_is_not_rounded(rows, cols, wdt):
    """dy that bf16 cannot hold, with an fp32 weight whose gradient shows it; by the call and through the graph."""
    torch = _torch()
    x, r = _randn((rows, cols), "bfloat16", 1), _randn((rows, cols), "bfloat16", 2)
    w = None if wdt is None else _randn((cols,), wdt, 3) + 1
    dy, dh = _randn((rows, cols), "float32", 4, 0.1), _randn((rows, cols), "bfloat16", 5, 0.1)
    h = (x.float() + r.float()).bfloat16()
    dx, dw = moe.moe_rms_norm_grad(dy, h, w, dh=dh)
    assert dx.dtype == torch.bfloat16 and (dw is None) == (w is None)
    _check(dx, dw, dy, h, w, dh)
    assert torch.equal(moe.moe_rms_norm_grad(dy, h, w, dh=dh.clone(), out=dh.clone())[0], dx)
    leaves = [t.requires_grad_() for t in (x, r, w) if t is not None]
    y, hh = moe.moe_rms_norm(x, w, residual=r, y_dtype=moe.MOE_F32)
    grads = torch.autograd.grad((y, hh), leaves, (dy, dh))
    assert torch.equal(grads[0], dx) and torch.equal(grads[1], dx) and (w is None or torch.equal(grads[2], dw))


def test_an_fp32_gradient_unaligned_in_place_and_refused():
    torch = _torch()
    flat = [_randn((9 * 65 + 1,), t, i) for i, t in enumerate(("float32", "bfloat16", "bfloat16"))]
    dy, h, dh = (f[1:].view(9, 65) for f in flat)
    dx, _ = moe.moe_rms_norm_grad(dy, h, dh=dh)
    _check(dx, None, dy, h, None, dh)
    assert torch.equal(moe.moe_rms_norm_grad(dy, h, dh=dh, out=dh)[0], dx)
    for bad in (lambda: moe.moe_rms_norm_grad(dy, h, out=dy), lambda: moe.moe_rms_norm_grad(dy.half(), h),
                lambda: moe.moe_rms_norm_grad(dy.double(), h), lambda: moe.moe_rms_norm_grad(dy[:8], h),
                lambda: moe.moe_rms_norm_grad(dy, h, dh=dy)):
        with pytest.raises(ValueError):
            bad()


def test_outputs_over_a_saved_tensor_are_noticed():
    """The first norm saved h1 for its backward pass, and the second writes its own h over it."""
    torch = _torch()
    x, w = _randn((5, 96), "float32", 1).requires_grad_(), _randn((96,), "float32", 2).requires_grad_()
    y1, h1 = moe.moe_rms_norm(x, w, residual=_randn((5, 96), "float32", 3))
    buffer = h1.detach()
    moe.moe_rms_norm(_randn((5, 96), "float32", 4), residual=buffer, h_out=buffer)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y1.sum().backward()
    y2 = moe.moe_rms_norm(x, w)
    with torch.no_grad():
        moe.moe_rms_norm(x, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y2.sum().backward()


def test_every_given_output_is_a_new_version():
    """Outputs of the norm, the conversions and the products; a new output is at version 0, what is only read stays."""
    torch = _torch()
    f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    b = lambda *s: torch.zeros(s, device="cuda", dtype=torch.uint8)  # noqa: E731
    i8 = lambda *s: torch.zeros(s, device="cuda", dtype=torch.int8)  # noqa: E731
    x, w, r, off = f(4, 64), f(64), f(4, 64), torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    w3, c, s, wc, ws = f(1, 8, 64), b(4, 32), b(4, 16), b(1, 8, 32), b(1, 8, 16)
    calls = [(lambda o: moe.moe_rms_norm(x, w, out=o), f(4, 64)),
             (lambda o: moe.moe_rms_norm(x, w, residual=r, h_out=o), f(4, 64)),
             (lambda o: moe.moe_rms_norm_i8(x, w, codes=o), i8(4, 64)), (lambda o: moe.moe_rms_norm_i8(x, w, scales=o), f(4)),
             (lambda o: moe.moe_rms_norm_i8(x, w, residual=r, h_out=o), f(4, 64)),
             (lambda o: moe.moe_rms_norm_grad(x, r, w, out=o), f(4, 64)),
             (lambda o: moe.moe_rms_norm_grad(x, r, w, dw_out=o), f(64)),
             (lambda o: moe.moe_quantize_rows(x, codes=o), i8(4, 64)), (lambda o: moe.moe_quantize_rows(x, scales=o), f(4)),
             (lambda o: moe.moe_quantize_mx4(x, codes=o), b(4, 32)), (lambda o: moe.moe_quantize_mx4(x, scales=o), b(4, 16)),
             (lambda o: moe.moe_dequantize_mx4(c, s, out=o), f(4, 64)),
             (lambda o: moe.moe_matmul_mx4(c, s, wc, ws, out=o), f(4, 8)),
             (lambda o: moe.moe_matmul_i8(i8(4, 64), f(4), i8(1, 8, 64), f(1, 8), out=o), f(4, 8)),
             (lambda o: moe.moe_grouped_matmul(x, w3, off, out=o), f(4, 8)),
             (lambda o: moe.moe_grouped_matmul_dx(f(4, 8), w3, off, out=o), f(4, 64)),
             (lambda o: moe.moe_grouped_matmul_dw(f(4, 8), x, off, out=o), f(1, 8, 64))]
    for i, (call, out) in enumerate(calls):
        before = out._version
        call(out)
        assert out._version > before, i
    assert all(t._version == 0 for t in (x, w, r, w3, c, s, wc, ws))
    assert all(t._version == 0 for t in moe.moe_rms_norm(x, w, residual=r))
    with torch.inference_mode():  # tensors without versions
        moe.moe_rms_norm(f(4, 64), out=f(4, 64))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_squares_outside_fp32(dtype):
    """Rows whose squares vanish or overflow, as include/moe.h states them; other rows keep their bits."""
    torch = _torch()
    x = _randn((5, 520), dtype, 1)
    plain = {eps: moe.moe_rms_norm(x, eps=eps) for eps in (0.0, 1e-6)}
    x[1], x[2], x[3] = 1e-23, 1e25, 0
    x[1, 0] = 0
    y = moe.moe_rms_norm(x, eps=0.0)
    assert bool(y[1, 0].isnan()) and bool((y[1, 1:] == float("inf")).all())
    assert not bool(y[2].any()) and bool(y[3].isnan().all())
    z = moe.moe_rms_norm(x, eps=1e-6)
    ref = x[1].double() * 1e3
    assert bool(((z[1].double() - ref).abs() <= (torch.finfo(x.dtype).eps / 2 + 40 * U) * ref).all())
    assert not bool(z[2].any()) and not bool(z[3].any())
    for i in (0, 4):
        assert torch.equal(y[i], plain[0.0][i]) and torch.equal(z[i], plain[1e-6][i])


@pytest.mark.parametrize("rows,cols", [(8191, 512), (8192, 512), (9003, 511), (8200, 385), (8200, 384), (8193, 383), (20000, 500)])
def test_gradients_of_many_narrow_fp32_rows(rows, cols):
    """On both sides of where 64 lanes take a row instead of 16; the same bits every time."""
    torch = _torch()
    dy, h, dh = (_randn((rows, cols), "float32", i, 0.5) for i in range(3))
    w = _randn((cols,), "bfloat16", 4) + 1
    dx, dw = moe.moe_rms_norm_grad(dy, h, w, dh=dh, dw_dtype=moe.MOE_F32)
    _check(dx, dw, dy, h, w, dh)
    again = moe.moe_rms_norm_grad(dy, h, w, dh=dh, dw_dtype=moe.MOE_F32)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
