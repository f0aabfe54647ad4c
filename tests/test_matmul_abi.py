"""The grouped products' C entries without a GPU: argument errors come back before anything is launched."""
import ctypes

import pytest

import moe_layer_forward_amd as moe

FAKE = ctypes.c_void_p(0x1000)
NULL = None


def _forward(dtype=1, G=2, N=64, K=64, off=FAKE, rows=10, x=FAKE, x_rows=10, idx=NULL, w=FAKE, y=FAKE, ydt=1, ws=FAKE,
             nb=1 << 40):
    return moe.load_library().moe_grouped_matmul(dtype, G, N, K, off, rows, x, x_rows, idx, w, y, ydt, ws, nb, None)


def _dx(dtype=1, G=2, N=64, K=64, off=FAKE, rows=10, dy=FAKE, w=FAKE, dx=FAKE, odt=1, ws=FAKE, nb=1 << 40):
    return moe.load_library().moe_grouped_matmul_dx(dtype, G, N, K, off, rows, dy, w, dx, odt, ws, nb, None)


def _dw(dtype=1, G=2, N=64, K=64, off=FAKE, rows=10, dy=FAKE, x=FAKE, x_rows=10, idx=NULL, dw=FAKE, odt=1, ws=FAKE,
        nb=1 << 40):
    return moe.load_library().moe_grouped_matmul_dw(dtype, G, N, K, off, rows, dy, x, x_rows, idx, dw, odt, ws, nb,
                                                    None)


def _i8(G=2, N=64, K=64, off=FAKE, rows=10, x=FAKE, xs=FAKE, x_rows=10, idx=NULL, w=FAKE, wsc=FAKE, y=FAKE, ydt=1,
        ws=FAKE, nb=1 << 40):
    return moe.load_library().moe_matmul_i8(G, N, K, off, rows, x, xs, x_rows, idx, w, wsc, y, ydt, ws, nb, None)


def _quant(dt=1, rows=4, cols=64, swiglu=0, x=FAKE, c=FAKE, s=FAKE):
    return moe.load_library().moe_quantize_rows(dt, rows, cols, swiglu, x, c, s, None)


INVALID, UNSUPPORTED = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
ODD = ctypes.c_void_p(0x1001)


@pytest.mark.parametrize("call", [_forward, _dx, _dw, _i8], ids=["forward", "dx", "dw", "i8"])
@pytest.mark.parametrize("args,status", [
    (dict(G=0), INVALID), (dict(G=5000), INVALID), (dict(N=0), INVALID), (dict(K=-1), INVALID),
    (dict(rows=-1), INVALID), (dict(off=NULL), INVALID), (dict(rows=1 << 31, x_rows=1 << 31), UNSUPPORTED),
    (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(N=1 << 20, K=1 << 16), UNSUPPORTED),
    (dict(off=ODD), INVALID),
])
def test_sizes_that_every_product_refuses(call, args, status):
    if call is _dx:
        args = {k: v for k, v in args.items() if k != "x_rows"}
    assert call(**args) == status
    assert moe.moe_last_error()


@pytest.mark.parametrize("call,args,status", [
    (_forward, dict(dtype=3), UNSUPPORTED), (_forward, dict(ydt=5), UNSUPPORTED), (_forward, dict(x=NULL), INVALID),
    (_forward, dict(w=NULL), INVALID), (_forward, dict(y=NULL), INVALID), (_forward, dict(x_rows=9), INVALID),
    (_forward, dict(idx=FAKE, x_rows=0), INVALID), (_forward, dict(x=ODD), INVALID),
    (_forward, dict(idx=FAKE, x_rows=1 << 26), UNSUPPORTED),
    (_dx, dict(dtype=-1), UNSUPPORTED), (_dx, dict(dy=NULL), INVALID), (_dx, dict(dx=ODD), INVALID),
    (_dw, dict(dw=NULL), INVALID), (_dw, dict(rows=0, dw=NULL), INVALID), (_dw, dict(x=NULL), INVALID),
    (_dw, dict(odt=2), UNSUPPORTED),
    (_i8, dict(K=131072), UNSUPPORTED), (_i8, dict(xs=NULL), INVALID), (_i8, dict(wsc=ODD), INVALID),
    (_i8, dict(ydt=9), UNSUPPORTED),
    (_quant, dict(dt=2), UNSUPPORTED), (_quant, dict(rows=-1), INVALID), (_quant, dict(cols=0), INVALID),
    (_quant, dict(swiglu=2), INVALID), (_quant, dict(x=NULL), INVALID), (_quant, dict(s=ODD), INVALID),
    (_quant, dict(cols=(1 << 20) + 1), UNSUPPORTED), (_quant, dict(rows=1 << 40), UNSUPPORTED),
])
def test_arguments_that_are_refused(call, args, status):
    assert call(**args) == status
    assert moe.moe_last_error()


def test_no_rows_launch_nothing():
    for call in (_forward, _dx, _i8, _quant):
        assert call(rows=0) == moe.MOE_OK and moe.moe_last_error() == ""


def test_workspace_sizes_and_refusal():
    """The size a call asks for is the size it insists on."""
    size = moe.moe_matmul_workspace_size
    for op, call in ((moe.MOE_MATMUL_FORWARD, _forward), (moe.MOE_MATMUL_DX, _dx), (moe.MOE_MATMUL_DW, _dw),
                     (moe.MOE_MATMUL_I8, _i8)):
        for G, rows, N, K in ((1, 64, 128, 8192), (1, 5000, 128, 256), (2, 64, 18432, 7168), (384, 512, 7168, 2048)):
            n = size(op, moe.MOE_BF16, G, rows, N, K)
            assert n >= 0
            if n:
                more = {} if call is _dx else {"x_rows": rows}
                assert call(G=G, rows=rows, N=N, K=K, ws=NULL, nb=0, **more) == moe.MOE_ERR_WORKSPACE
                assert call(G=G, rows=rows, N=N, K=K, nb=n - 1, **more) == moe.MOE_ERR_WORKSPACE
                assert call(G=G, rows=rows, N=N, K=K, ws=ctypes.c_void_p(0x1010), nb=n, **more) == moe.MOE_ERR_WORKSPACE
    with pytest.raises(moe.MoeError):
        size(9, moe.MOE_BF16, 1, 1, 1, 1)
    with pytest.raises(moe.MoeError):
        size(moe.MOE_MATMUL_DX, 7, 1, 1, 1, 1)
    with pytest.raises(moe.MoeError):
        size(moe.MOE_MATMUL_I8, moe.MOE_F32, 1, 1, 1, 200000)
