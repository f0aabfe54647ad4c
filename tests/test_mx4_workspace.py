"""The microscaled product's workspace without a GPU: sizes that pack their scales insist on it."""
import ctypes

import pytest

import moe_layer_forward_amd as moe

FAKE, EIGHT = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)


def _call(G, rows, N, K, ws, nb):
    return moe.load_library().moe_matmul_mx4(G, N, K, FAKE, rows, FAKE, FAKE, rows, None, FAKE, FAKE, FAKE, 1, ws, nb, None)


@pytest.mark.parametrize("G,rows,N,K", [(1, 8192, 18432, 7168), (3, 3 * 16384, 4096, 7168), (1, 6111, 5103, 6176),
                                        (3, 8277, 5120, 6048)])
def test_packed_scales_need_their_workspace(G, rows, N, K):
    """Packed scales: those of every row tile of 256 and of every group's columns, 16 bytes a row and 512 values."""
    n = moe.moe_matmul_workspace_size(moe.MOE_MATMUL_MX4, moe.MOE_BF16, G, rows, N, K)
    assert n >= (rows + G * N) * moe.mx4_scale_cols(K)
    for ws, nb in ((FAKE, n - 1), (FAKE, 0), (None, n), (None, 0), (EIGHT, n)):
        assert _call(G, rows, N, K, ws, nb) == moe.MOE_ERR_WORKSPACE and moe.moe_last_error(), (ws, nb)


@pytest.mark.parametrize("G,rows,N,K", [(1, 64, 128, 8192), (384, 512, 7168, 2048), (48, 8192, 2048, 7168), (1, 0, 64, 64)])
def test_other_sizes_need_none(G, rows, N, K):
    assert moe.moe_matmul_workspace_size(moe.MOE_MATMUL_MX4, moe.MOE_BF16, G, rows, N, K) == 0
