"""The norm's C entries and binding without a GPU: what is refused before anything is launched."""
import ctypes

import pytest

import moe_layer_forward_amd as moe

FAKE, TWO, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1002), ctypes.c_void_p(0x1001)
INVALID, WORKSPACE = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("dtype,dy,h,ws,status", [
    (moe.MOE_BF16, TWO, FAKE, FAKE, INVALID),  # an fp32 dy on 2 bytes
    (moe.MOE_F32, TWO, FAKE, FAKE, INVALID), (moe.MOE_BF16, FAKE, ODD, FAKE, INVALID),
    (moe.MOE_BF16, None, FAKE, FAKE, INVALID), (moe.MOE_BF16, FAKE, TWO, None, WORKSPACE), (7, FAKE, FAKE, FAKE, None)])
def test_gradient_of_an_fp32_y(dtype, dy, h, ws, status):
    got = moe.load_library().moe_rms_norm_grad_f32(dtype, 4, 64, dy, h, FAKE, 1, 1e-6, None, FAKE, FAKE, 1, ws, 1 << 30,
                                                   None)
    assert got == (moe.MOE_ERR_UNSUPPORTED if status is None else status)
    assert "moe_rms_norm_grad_f32" in moe.moe_last_error() or status == WORKSPACE


def test_dual_tensors_are_refused():
    """Forward-mode derivatives: the tangent of a dual tensor, which asks for no gradient, would be lost."""
    torch = pytest.importorskip("torch")
    forward_ad = torch.autograd.forward_ad
    x, w, w3 = torch.ones(4, 64), torch.ones(64), torch.ones(1, 8, 64)
    with forward_ad.dual_level():
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        for call in (lambda: moe.moe_rms_norm(dual(x), w), lambda: moe.moe_rms_norm(x, dual(w)),
                     lambda: moe.moe_rms_norm(x, w, residual=dual(x)), lambda: moe.moe_rms_norm(dual(x), out=x),
                     lambda: moe.moe_grouped_matmul(dual(x), w3, None), lambda: moe.moe_grouped_matmul(x, dual(w3), None)):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
        with pytest.raises(ValueError, match="GPU"):  # no tangent: the call goes on to its other checks
            moe.moe_rms_norm(x, w)


def test_leaves_outside_the_gpu_are_refused_like_every_tensor():
    torch = pytest.importorskip("torch")
    x, w = torch.ones(4, 64), torch.ones(64)
    for args in ((x, w), (x.clone().requires_grad_(), w), (x, w.clone().requires_grad_())):
        with pytest.raises(ValueError, match="every tensor must live on the GPU"):
            moe.moe_rms_norm(*args)


def test_h_and_y_in_one_place_are_refused():
    """Each may be x, but one would overwrite the other."""
    lib, y = moe.load_library(), ctypes.c_void_p(0x2000)
    assert lib.moe_rms_norm(1, 4, 64, FAKE, FAKE, FAKE, 1, 1e-6, FAKE, FAKE, 1, None) == INVALID
    assert "same" in moe.moe_last_error()
    assert lib.moe_rms_norm_i8(1, 4, 64, FAKE, FAKE, FAKE, 1, 1e-6, y, y, FAKE, None) == INVALID
    assert "same" in moe.moe_last_error()
