"""The root-mean-square norm, its 8-bit output and its gradients against float64.

u = 2^-24 is half a step of fp32.  A row's sum of squares is a chain of at most 40 additions in a lane and 22 over the
lanes, so 1 / sqrt of it is off by at most (62 + 1) / 2 + 4 u, and y, two products later, by less than 40 u and the
rounding of its type."""
import numpy as np
import pytest

import moe_layer_forward_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
COLS = (1, 7, 8, 9, 64, 511, 513, 1001, 2048, 2049, 4096, 7168, 8192, 8193, 12288, 18432, 32768)


def _torch():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def _type(dt):
    torch = _torch()
    return {"bf16": torch.bfloat16, "f32": torch.float32}[dt]


def _randn(shape, dt, seed, scale=1.0):
    torch = _torch()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(_type(dt))


def _reference(h, w, eps):
    """y in float64"""
    h = h.double()
    y = h / ((h * h).mean(dim=1, keepdim=True) + eps).sqrt()
    return y if w is None else y * w.double()


def _check_y(y, ref, dt):
    err = (y.double() - ref).abs()
    bound = (HALF[dt] + 40 * U) * ref.abs() + 2.0 ** -126
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dt,wdt,ydt", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f32", "f32", "f32"), ("f32", "bf16", "bf16")])
def test_norm_of_the_sum(cols, dt, wdt, ydt):
    torch = _torch()
    for rows in (1, 5):
        x, r = _randn((rows, cols), dt, 1), _randn((rows, cols), dt, 2, 5.0)
        w = _randn((cols,), wdt, 3) + 1
        y, h = moe.moe_rms_norm(x, w, residual=r, eps=1e-5, y_dtype=moe.MOE_BF16 if ydt == "bf16" else moe.MOE_F32)
        assert torch.equal(h, (x.float() + r.float()).to(h.dtype))
        assert y.dtype == _type(ydt)
        _check_y(y, _reference(h, w, 1e-5), ydt)
        q, s, h8 = moe.moe_rms_norm_i8(x, w, residual=r, eps=1e-5)
        assert torch.equal(h, h8)
        _check_codes(q, s, _reference(h, w, 1e-5))


def _check_codes(q, s, ref):
    """Codes are off by half a step, and by what y and its largest value are off: 127 * 2 * 42 u < 1e-3."""
    a = ref.abs().amax(dim=1)
    assert bool(((s.double() - a / 127).abs() <= 44 * U * a / 127 + 2.0 ** -126).all())
    t = 127 * ref / a.clamp(min=1e-300)[:, None]
    assert bool(((q.double() - t).abs() <= 0.5 + 1e-3).all())


@pytest.mark.parametrize("rows,cols", [(2, 300), (1, 7168), (300, 7168), (64, 7168), (4097, 1024), (20000, 136), (3, 20000),
                                       (9001, 511), (8193, 257), (513, 5), (1111, 128), (700, 256)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_without_residual_or_weight(rows, cols, dt):
    x, w = _randn((rows, cols), dt, rows), _randn((cols,), dt, 7)
    _check_y(moe.moe_rms_norm(x, w), _reference(x, w, 1e-6), dt)
    _check_y(moe.moe_rms_norm(x, eps=0.0), _reference(x, None, 0.0), dt)
    _check_codes(*moe.moe_rms_norm_i8(x), _reference(x, None, 1e-6))


@pytest.mark.parametrize("cols", [65, 4096, 20001])
def test_rows_that_start_anywhere_and_outputs_in_place(cols):
    torch = _torch()
    for dt in ("bf16", "f32"):
        flat, rflat, w = _randn((7 * cols + 3,), dt, 1), _randn((7 * cols + 1,), dt, 2), _randn((cols + 1,), dt, 3)[1:]
        x, r = flat[3:].view(7, cols), rflat[1:].view(7, cols)
        want_y, want_h = moe.moe_rms_norm(x.clone(), w.clone(), residual=r.clone())
        x1, r1 = flat.clone()[3:].view(7, cols), rflat.clone()[1:].view(7, cols)
        y, h = moe.moe_rms_norm(x1, w, residual=r1, out=x1, h_out=r1)
        assert y is x1 and h is r1 and torch.equal(y, want_y) and torch.equal(h, want_h)
        want = moe.moe_rms_norm(x.clone(), w)
        x1 = flat.clone()[3:].view(7, cols)
        assert torch.equal(moe.moe_rms_norm(x1, w, out=x1), want)
        q, s, h = moe.moe_rms_norm_i8(x, w, residual=r, h_out=r)
        assert h is r and torch.equal(r, want_h)
        q2, s2 = moe.moe_rms_norm_i8(want_h, w)
        assert torch.equal(q, q2) and torch.equal(s, s2)


def test_zeros_infinities_and_nan_stay_in_their_row():
    torch = _torch()
    x = _randn((6, 515), "bf16", 1)
    plain = moe.moe_rms_norm(x)
    q0, s0 = moe.moe_rms_norm_i8(x)
    x[1] = 0
    x[3, 514] = float("nan")
    x[4, 2] = float("inf")
    y = moe.moe_rms_norm(x)
    q, s = moe.moe_rms_norm_i8(x)
    for i in (0, 2, 5):
        assert torch.equal(y[i], plain[i]) and torch.equal(q[i], q0[i]) and torch.equal(s[i], s0[i])
    assert not bool(y[1].any()) and not bool(q[1].any()) and float(s[1]) == 0
    assert bool(y[3].isnan().all()) and bool(y[4, 2].isnan()) and not bool(y[4, 3:].any())
    assert bool(s[3:5].isnan().all()) and not bool(q[3:5].any())


@pytest.mark.parametrize("rows,cols", [(9001, 511), (515, 200), (1111, 128), (8200, 320), (600, 7)])
@pytest.mark.parametrize("dt,wdt", [("bf16", "f32"), ("f32", "bf16")])
def test_many_short_rows(rows, cols, dt, wdt):
    """With a residual, at any alignment, in place: h and y of a few rows more and of the rows themselves."""
    torch = _torch()
    flat = [_randn((rows * cols + 1,), dt, i) for i in range(2)]
    x, r = (f[1:].view(rows, cols) for f in flat)
    w = _randn((cols,), wdt, 3)
    want_h = (x.float() + r.float()).to(x.dtype)
    ref = _reference(want_h, w, 1e-5)
    q, s, h = moe.moe_rms_norm_i8(x, w, residual=r, eps=1e-5)
    assert torch.equal(h, want_h)
    _check_codes(q, s, ref)
    y, h = moe.moe_rms_norm(x, w, residual=r, eps=1e-5, out=x, h_out=r)
    assert y is x and h is r and torch.equal(r, want_h) and float(flat[1][0]) == float(_randn((rows * cols + 1,), dt, 1)[0])
    _check_y(y, ref, dt)


def test_no_rows_and_a_row_of_one():
    torch = _torch()
    x, w = torch.empty((0, 128), device="cuda"), torch.ones(128, device="cuda")
    assert moe.moe_rms_norm(x, w).shape == (0, 128)
    dx, dw = moe.moe_rms_norm_grad(x, x, w)
    assert dx.shape == (0, 128) and not bool(dw.any())
    one = torch.tensor([[-3.0]], device="cuda")
    assert float(moe.moe_rms_norm(one, eps=0.0)) == -1.0


def _grad_reference(dy, h, w, dh, eps):
    """(dx, dw) in float64, and the magnitudes their errors are relative to."""
    torch = _torch()
    dy, h = dy.double(), h.double()
    w = torch.ones(h.shape[1], device="cuda", dtype=torch.float64) if w is None else w.double()
    n = h.shape[1]
    m = 1 / ((h * h).mean(dim=1, keepdim=True) + eps).sqrt()
    g = dy * w
    dx = m * (g - h * m ** 2 * (g * h).sum(dim=1, keepdim=True) / n)
    mag = m * (g.abs() + h.abs() * m ** 2 * (g * h).abs().sum(dim=1, keepdim=True) / n)
    if dh is not None:
        dx, mag = dx + dh.double(), mag + dh.double().abs()
    return dx, mag, (dy * h * m).sum(dim=0), (dy * h * m).abs().sum(dim=0)


def _check_grads(dx, dw, dy, h, w, dh, eps, dt, wdt):
    """dx: two sums of 64 roundings each and a handful of products, 160 u of the magnitudes, and one rounding.  dw: 40 u a
    term, a chain of at most rows / 128 terms in a work-group and 150 after it."""
    rdx, mag, rdw, wmag = _grad_reference(dy, h, w, dh, eps)
    err = (dx.double() - rdx).abs()
    bound = 160 * U * mag + HALF[dt] * rdx.abs() + 2.0 ** -126
    assert bool((err <= bound).all()), float((err / bound).max())
    if dw is not None:
        err = (dw.double() - rdw).abs()
        bound = (190 + h.shape[0] / 128) * U * wmag + HALF[wdt] * rdw.abs() + 2.0 ** -126
        assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dt,wdt", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
def test_gradients(cols, dt, wdt):
    for rows, with_dh in ((1, True), (6, False), (530, True)):
        dy, h, w = _randn((rows, cols), dt, 1, 0.1), _randn((rows, cols), dt, 2, 3.0), _randn((cols,), wdt, 3) + 1
        dh = _randn((rows, cols), dt, 4, 0.1) if with_dh else None
        dx, dw = moe.moe_rms_norm_grad(dy, h, w, dh=dh, eps=1e-5)
        assert dw.dtype == _type(wdt)
        _check_grads(dx, dw, dy, h, w, dh, 1e-5, dt, wdt)


@pytest.mark.parametrize("rows,cols", [(5000, 72), (515, 9), (9003, 511), (777, 128), (3001, 2048), (2500, 4104), (1500, 10000)])
def test_gradients_of_many_rows_are_the_same_every_time(rows, cols):
    torch = _torch()
    dy, h, w = _randn((rows, cols), "bf16", 1), _randn((rows, cols), "bf16", 2), _randn((cols,), "f32", 3)
    dx, dw = moe.moe_rms_norm_grad(dy, h, w)
    _check_grads(dx, dw, dy, h, w, None, 1e-6, "bf16", "f32")
    for _ in range(3):
        dx2, dw2 = moe.moe_rms_norm_grad(dy, h, w)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_gradients_in_place_unaligned_and_without_a_weight():
    torch = _torch()
    for cols in (65, 5000, 12345):
        flat = [_randn((9 * cols + 1,), "bf16", i) for i in range(3)]
        dy, h, dh = (f[1:].view(9, cols) for f in flat)
        dx, dw = moe.moe_rms_norm_grad(dy.clone(), h.clone(), dh=dh.clone())
        assert dw is None
        _check_grads(dx, None, dy, h, None, dh, 1e-6, "bf16", None)
        over = dy.clone()
        assert torch.equal(moe.moe_rms_norm_grad(over, h, dh=dh, out=over)[0], dx)
        assert torch.equal(moe.moe_rms_norm_grad(dy, h, dh=dh, out=dh)[0], dx)


def test_gradients_against_differences():
    """(f(x + d v) - f(x - d v)) / 2 d in fp32, f a weighted sum of y and h, v the gradient's direction or any.  Each f is
    off by 42 u of its terms' magnitudes, over d; the difference by d^2 f''' / 6, where f changes over lengths of |h| (27
    here, a row's 13): less than d^2 |grad| / 100."""
    torch = _torch()
    rows, cols, d = 4, 96, 2.0 ** -4
    args = [_randn(s, "f32", i) for i, s in enumerate(((rows, cols), (rows, cols), (cols,)))]
    cy, ch = _randn((rows, cols), "f32", 8).double(), _randn((rows, cols), "f32", 9).double()

    def f(x, r, w):
        y, h = moe.moe_rms_norm(x, w, residual=r)
        return (y.double() * cy).sum() + (h.double() * ch).sum(), (y.double() * cy).abs().sum() + (h.double() * ch).abs().sum()

    grads = torch.autograd.grad(f(*(a.requires_grad_() for a in args))[0], args)
    args = [a.detach() for a in args]
    for i, grad in enumerate(grads):
        for seed in range(3):
            v = grad if seed == 0 else _randn(grad.shape, "f32", 20 + seed)
            v = v.double() / v.double().norm()
            up, down = list(args), list(args)
            up[i], down[i] = (args[i] + d * v).float(), (args[i] - d * v).float()
            step = float(((up[i].double() - down[i].double()) * grad.double()).sum())
            diff = float(f(*up)[0] - f(*down)[0])
            bound = 2 * 42 * U * float(f(*args)[1]) + 2 * d ** 3 * float(grad.norm()) / 100
            assert abs(diff - step) < bound, (i, seed, diff, step, bound)


@pytest.mark.parametrize("dt,wdt", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
def test_torch_graph(dt, wdt):
    torch = _torch()
    x, r, w = (_randn(s, t, i).requires_grad_() for i, (s, t) in enumerate((((33, 200), dt), ((33, 200), dt), ((200,), wdt))))
    cy, ch = _randn((33, 200), dt, 5), _randn((33, 200), dt, 6)
    y, h = moe.moe_rms_norm(x, w, residual=r)
    torch.autograd.backward((y, h), (cy, ch))
    dx, dw = moe.moe_rms_norm_grad(cy, h.detach(), w.detach(), dh=ch)
    assert torch.equal(x.grad, dx) and torch.equal(r.grad, dx) and torch.equal(w.grad, dw)
    # only one of the outputs is used; only one of the inputs asks
    (gx,) = torch.autograd.grad(moe.moe_rms_norm(x, w, residual=r)[1], (x,), ch)
    assert torch.equal(gx, ch)
    (gw,) = torch.autograd.grad(moe.moe_rms_norm(x.detach(), w), (w,), cy)
    assert torch.equal(gw, moe.moe_rms_norm_grad(cy, x.detach(), w.detach())[1])
    (gr,) = torch.autograd.grad(moe.moe_rms_norm(x.detach(), w.detach(), residual=r)[0], (r,), cy)
    assert torch.equal(gr, moe.moe_rms_norm_grad(cy, h.detach(), w.detach())[0])
    # an fp32 y of bf16 rows, and a gradient that is not contiguous
    y = moe.moe_rms_norm(x, w, y_dtype=moe.MOE_F32)
    (gx,) = torch.autograd.grad(y.t(), (x,), cy.float().t().contiguous())
    assert torch.equal(gx, moe.moe_rms_norm_grad(cy, x.detach(), w.detach())[0])
    # nothing asks, or the result goes to a given place: no graph
    with torch.no_grad():
        assert not moe.moe_rms_norm(x, w).requires_grad
    assert not moe.moe_rms_norm(x, w, out=torch.empty_like(x)).requires_grad
    assert not moe.moe_rms_norm(x.detach(), w.detach()).requires_grad


def test_another_stream_and_a_captured_graph():
    """Replays of a norm with its gradients, new inputs in between, against eager calls."""
    torch = _torch()
    rows, cols = 300, 1000
    x, r, w, dy = _randn((rows, cols), "bf16", 1), _randn((rows, cols), "bf16", 2), _randn((cols,), "f32", 3), _randn((rows, cols), "bf16", 4)
    ws = torch.empty(moe.moe_rms_norm_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")

    def run():
        y, h = moe.moe_rms_norm(x, w, residual=r)
        q, s = moe.moe_rms_norm_i8(y, w)
        return (y, h, q, s, *moe.moe_rms_norm_grad(dy, h, w, dh=y, workspace=ws))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, run()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in range(4):
        for t, k in ((x, 1), (r, 2), (dy, 3)):
            t.copy_(_randn(t.shape, "bf16", 10 * seed + k))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, run()))


def test_refusals():
    torch = _torch()
    x, w = torch.zeros((4, 64), device="cuda"), torch.ones(64, device="cuda")
    for bad in (lambda: moe.moe_rms_norm(x.half(), w), lambda: moe.moe_rms_norm(x, w[:63]), lambda: moe.moe_rms_norm(x[0], w),
                lambda: moe.moe_rms_norm(x, w, residual=x.bfloat16()), lambda: moe.moe_rms_norm(x, w, residual=x[:3]),
                lambda: moe.moe_rms_norm(x, w, h_out=x), lambda: moe.moe_rms_norm(x[:, ::2], w[:32]),
                lambda: moe.moe_rms_norm(x.t(), w[:4]), lambda: moe.moe_rms_norm(x, w.cpu()),
                lambda: moe.moe_rms_norm(x, w, out=x.bfloat16()[:2]), lambda: moe.moe_rms_norm(x, w, y_dtype=9),
                lambda: moe.moe_rms_norm_i8(x, w, codes=torch.zeros((4, 64), device="cuda")),
                lambda: moe.moe_rms_norm_i8(x, w, scales=torch.zeros(5, device="cuda")),
                lambda: moe.moe_rms_norm_grad(x.bfloat16(), x, w), lambda: moe.moe_rms_norm_grad(x, x, w, dh=x[:2]),
                lambda: moe.moe_rms_norm_grad(x, x, dw_out=w), lambda: moe.moe_rms_norm_grad(x, x, w, need_dw=False, dw_out=w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: moe.moe_rms_norm(x, w, eps=-1.0), lambda: moe.moe_rms_norm(torch.zeros((1, 32769), device="cuda")),
                lambda: moe.moe_rms_norm_grad(x, x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(moe.MoeError):
            bad()
    assert not np.any(x.cpu().numpy())


@pytest.mark.parametrize("rows,cols", [(5300, 7168), (20000, 2048), (8000, 14336)])
def test_large_matrices(rows, cols):
    """Sizes that move with the non-temporal policy, y too in the last."""
    torch = _torch()
    x, r, w = _randn((rows, cols), "bf16", 1), _randn((rows, cols), "bf16", 2), _randn((cols,), "f32", 3)
    y, h = moe.moe_rms_norm(x, w, residual=r)
    assert torch.equal(h, (x.float() + r.float()).bfloat16())
    ref = _reference(h, w, 1e-6)
    _check_y(y, ref, "bf16")
    q, s, h8 = moe.moe_rms_norm_i8(x, w, residual=r)
    assert torch.equal(h, h8)
    _check_codes(q, s, ref)
    del ref, q, s, h8
    dx, dw = moe.moe_rms_norm_grad(x, h, w, dh=r)
    _check_grads(dx, dw, x, h, w, r, 1e-6, "bf16", "f32")


def test_a_captured_backward_pass():
    """Forward and backward in one graph, against eager calls; refused while an eager graph of the same leaves lives."""
    torch = _torch()
    x, r, w = (_randn(s, t, i).requires_grad_() for i, (s, t) in enumerate((((40, 520), "bf16"), ((40, 520), "bf16"), ((520,), "f32"))))
    cy, ch = _randn((40, 520), "bf16", 5), _randn((40, 520), "bf16", 6)

    def step():
        y, h = moe.moe_rms_norm(x, w, residual=r)
        return torch.autograd.grad((y, h), (x, r, w), (cy, ch))

    alive = moe.moe_rms_norm(x, w, residual=r)
    with pytest.raises(RuntimeError, match="same leaves"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            torch.zeros(1, device="cuda")
            moe.moe_rms_norm(x, w, residual=r)
    del alive
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for seed in range(4):
        with torch.no_grad():
            x.copy_(_randn(x.shape, "bf16", 30 + seed))
            w.copy_(_randn(w.shape, "f32", 40 + seed))
            cy.copy_(_randn(cy.shape, "bf16", 50 + seed))
        graph.replay()
        torch.cuda.synchronize()
        h = (x.detach().float() + r.detach().float()).bfloat16()
        dx, dw = moe.moe_rms_norm_grad(cy, h, w.detach(), dh=ch)
        assert torch.equal(out[0], dx) and torch.equal(out[1], dx) and torch.equal(out[2], dw)


def test_past_four_gib():
    """The last rows of matrices of 5.6 GB are those of small calls."""
    torch = _torch()
    rows, cols = 700000, 4000
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-4:] = _randn((4, cols), "bf16", 1)
    w = _randn((cols,), "bf16", 2)
    y, h = moe.moe_rms_norm(x, w, residual=x)
    small_y, small_h = moe.moe_rms_norm(x[-4:], w, residual=x[-4:])
    assert torch.equal(h[-4:], small_h) and not bool(y[:-4].any())
    _check_y(y[-4:], _reference(small_h, w, 1e-6), "bf16")
    _check_y(small_y, _reference(small_h, w, 1e-6), "bf16")
    q, s = moe.moe_rms_norm_i8(x, w)
    q2, s2 = moe.moe_rms_norm_i8(x[-4:], w)
    assert bool((q[-4:].int() - q2.int()).abs().max() <= 1) and torch.allclose(s[-4:], s2, rtol=1e-5) and not bool(q[:-4].any())
    dx, dw = moe.moe_rms_norm_grad(y, h, w, out=y)
    small_dx, small_dw = moe.moe_rms_norm_grad(small_y.clone(), small_h, w)
    assert bool(((dx[-4:].float() - small_dx.float()).abs() <= 0.02 * small_dx.float().abs().max()).all())
    assert bool(((dw.float() - small_dw.float()).abs() <= 0.01 * small_dw.float().abs() + 1e-3 * small_dw.float().abs().max()).all())
