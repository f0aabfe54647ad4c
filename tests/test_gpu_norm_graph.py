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
