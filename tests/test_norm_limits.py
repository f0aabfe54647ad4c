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
