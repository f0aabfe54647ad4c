"""The norm's and the microscaled 4-bit C entries without a GPU: argument errors come back before anything is launched."""
import ctypes

import pytest

import moe_layer_forward_amd as moe

FAKE, ODD, EIGHT, NULL = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1001), ctypes.c_void_p(0x1008), None
INVALID, UNSUPPORTED, WORKSPACE = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


def _norm(dt=1, rows=4, cols=64, x=FAKE, r=NULL, w=FAKE, wdt=1, eps=1e-6, h=NULL, y=FAKE, ydt=1):
    return moe.load_library().moe_rms_norm(dt, rows, cols, x, r, w, wdt, eps, h, y, ydt, None)


def _norm8(dt=1, rows=4, cols=64, x=FAKE, r=NULL, w=FAKE, wdt=1, eps=1e-6, h=NULL, y=FAKE, s=FAKE):
    return moe.load_library().moe_rms_norm_i8(dt, rows, cols, x, r, w, wdt, eps, h, y, s, None)


def _grad(dt=1, rows=4, cols=64, dy=FAKE, x=FAKE, w=FAKE, wdt=1, eps=1e-6, dh=NULL, y=FAKE, dw=FAKE, dwt=1, ws=FAKE,
          nb=1 << 40):
    return moe.load_library().moe_rms_norm_grad(dt, rows, cols, dy, x, w, wdt, eps, dh, y, dw, dwt, ws, nb, None)


def _quant(dt=1, rows=4, cols=64, swiglu=0, x=FAKE, c=FAKE, s=FAKE):
    return moe.load_library().moe_quantize_mx4(dt, rows, cols, swiglu, x, c, s, None)


def _dequant(dt=1, rows=4, cols=64, c=FAKE, s=FAKE, x=FAKE):
    return moe.load_library().moe_dequantize_mx4(rows, cols, c, s, x, dt, None)


def _mx4(G=2, N=64, K=64, off=FAKE, rows=10, x=FAKE, xs=FAKE, x_rows=10, idx=NULL, w=FAKE, wsc=FAKE, y=FAKE, ydt=1,
         ws=FAKE, nb=1 << 40):
    return moe.load_library().moe_matmul_mx4(G, N, K, off, rows, x, xs, x_rows, idx, w, wsc, y, ydt, ws, nb, None)


@pytest.mark.parametrize("call", [_norm, _norm8, _grad], ids=["norm", "norm8", "grad"])
@pytest.mark.parametrize("args,status", [
    (dict(dt=2), UNSUPPORTED), (dict(wdt=-1), UNSUPPORTED), (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
    (dict(cols=32769), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED), (dict(eps=-1e-6), INVALID), (dict(eps=NAN), INVALID),
    (dict(eps=INF), INVALID), (dict(x=NULL), INVALID), (dict(y=NULL), INVALID), (dict(x=ODD), INVALID),
    (dict(w=ODD), INVALID), (dict(wdt=0, w=ctypes.c_void_p(0x1002)), INVALID),
])
def test_what_every_norm_refuses(call, args, status):
    assert call(**args) == status
    assert moe.moe_last_error()


@pytest.mark.parametrize("call,args,status", [
    (_norm, dict(ydt=7), UNSUPPORTED), (_norm, dict(r=FAKE), INVALID), (_norm, dict(h=FAKE), INVALID),
    (_norm, dict(r=ODD, h=FAKE), INVALID), (_norm, dict(r=FAKE, h=ODD), INVALID), (_norm, dict(y=ODD), INVALID),
    (_norm8, dict(s=NULL), INVALID), (_norm8, dict(s=ODD), INVALID), (_norm8, dict(r=FAKE), INVALID),
    (_grad, dict(dy=NULL), INVALID), (_grad, dict(dy=ODD), INVALID), (_grad, dict(dh=ODD), INVALID),
    (_grad, dict(dwt=3), UNSUPPORTED), (_grad, dict(dw=ODD), INVALID), (_grad, dict(ws=NULL), WORKSPACE),
    (_grad, dict(nb=0), WORKSPACE), (_grad, dict(ws=EIGHT), WORKSPACE),
    (_quant, dict(dt=2), UNSUPPORTED), (_quant, dict(rows=-1), INVALID), (_quant, dict(cols=0), INVALID),
    (_quant, dict(cols=48), INVALID), (_quant, dict(cols=(1 << 20) + 32), UNSUPPORTED), (_quant, dict(rows=1 << 40), UNSUPPORTED),
    (_quant, dict(swiglu=2), INVALID), (_quant, dict(x=NULL), INVALID), (_quant, dict(c=EIGHT), INVALID),
    (_quant, dict(s=EIGHT), INVALID), (_quant, dict(x=ODD), INVALID),
    (_dequant, dict(dt=5), UNSUPPORTED), (_dequant, dict(cols=33), INVALID), (_dequant, dict(c=NULL), INVALID),
    (_dequant, dict(x=ODD), INVALID), (_dequant, dict(s=ODD), INVALID),
    (_mx4, dict(G=0), INVALID), (_mx4, dict(G=4097), INVALID), (_mx4, dict(N=0), INVALID), (_mx4, dict(K=0), INVALID),
    (_mx4, dict(K=65), INVALID), (_mx4, dict(K=16), INVALID), (_mx4, dict(rows=-1), INVALID), (_mx4, dict(off=NULL), INVALID),
    (_mx4, dict(off=ODD), INVALID), (_mx4, dict(idx=ODD), INVALID), (_mx4, dict(ydt=4), UNSUPPORTED),
    (_mx4, dict(rows=1 << 31, x_rows=1 << 31), UNSUPPORTED), (_mx4, dict(N=(1 << 20) + 1), UNSUPPORTED),
    (_mx4, dict(K=(1 << 20) + 32), UNSUPPORTED), (_mx4, dict(N=1 << 20, K=1 << 13), UNSUPPORTED),
    (_mx4, dict(x_rows=9), INVALID), (_mx4, dict(idx=FAKE, x_rows=0), INVALID),
    (_mx4, dict(idx=FAKE, x_rows=1 << 28), UNSUPPORTED), (_mx4, dict(x=NULL), INVALID), (_mx4, dict(xs=NULL), INVALID),
    (_mx4, dict(w=EIGHT), INVALID), (_mx4, dict(wsc=EIGHT), INVALID), (_mx4, dict(xs=EIGHT), INVALID), (_mx4, dict(y=ODD), INVALID),
    (_mx4, dict(rows=(1 << 31) - 1, x_rows=(1 << 31) - 1, N=1 << 20), UNSUPPORTED),
])
def test_arguments_that_are_refused(call, args, status):
    assert call(**args) == status
    assert moe.moe_last_error()


def test_no_rows_launch_nothing():
    for call in (_norm, _norm8, _quant, _dequant, _mx4):
        assert call(rows=0) == moe.MOE_OK and moe.moe_last_error() == ""
    assert _grad(rows=0, dw=NULL) == moe.MOE_OK


def test_workspace_sizes_and_refusal():
    """The size a call asks for is the size it insists on."""
    for rows, cols in ((1, 1), (4, 64), (100, 7168), (16384, 7168), (7, 32768)):
        n = moe.moe_rms_norm_workspace_size(rows, cols)
        assert n >= 4 * cols and n % 256 == 0
        assert _grad(rows=rows, cols=cols, nb=n - 1) == WORKSPACE
    for G, rows, N, K in ((1, 64, 128, 8192), (1, 5000, 128, 256), (2, 64, 18432, 7168), (384, 512, 7168, 2048)):
        n = moe.moe_matmul_workspace_size(moe.MOE_MATMUL_MX4, moe.MOE_BF16, G, rows, N, K)
        if n:
            assert _mx4(G=G, rows=rows, x_rows=rows, N=N, K=K, nb=n - 1) == WORKSPACE
            assert _mx4(G=G, rows=rows, x_rows=rows, N=N, K=K, ws=NULL, nb=0) == WORKSPACE
    for bad in ((-1, 64), (4, 0), (4, 40000)):
        with pytest.raises(moe.MoeError):
            moe.moe_rms_norm_workspace_size(*bad)
    with pytest.raises(moe.MoeError):
        moe.moe_matmul_workspace_size(moe.MOE_MATMUL_MX4, moe.MOE_BF16, 1, 1, 64, 63)


def test_scale_cols():
    assert [moe.mx4_scale_cols(k) for k in (32, 512, 544, 2048, 7168, 18432)] == [16, 16, 32, 64, 224, 576]
