"""The grouped products' limits as include/moe.h states them, just inside and just outside (no GPU: refusals and
workspace sizes only; an accepted size is told from a refusal that comes later)."""
import ctypes

import pytest

import moe_layer_forward_amd as moe

FAKE, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1001)
FORWARD, DX, DW, I8 = moe.MOE_MATMUL_FORWARD, moe.MOE_MATMUL_DX, moe.MOE_MATMUL_DW, moe.MOE_MATMUL_I8
MOST = 2 ** 31 - 1


@pytest.mark.parametrize("op,G,rows,N,K", [
    (FORWARD, 1, 1 << 20, 32768, 64), (DW, 384, 8192, 18432, 7168), (DX, 4096, 4096, 8, 1 << 20),
    (FORWARD, 1, MOST, 4096, 8), (DX, 1, MOST, 8, 4096), (I8, 1, MOST, 4096, 8), (DW, 1, MOST, 8, 8),
    (DW, 4096, 0, 1 << 20, 1), (DW, 4096, 100, 1 << 16, (1 << 15) - 1), (I8, 1, 100, 65537, 65535),
    (FORWARD, 1, 100, 1 << 16, (1 << 15) - 1),
])
def test_sizes_inside_the_limits(op, G, rows, N, K):
    assert moe.moe_matmul_workspace_size(op, moe.MOE_BF16, G, rows, N, K) >= 0


@pytest.mark.parametrize("op,G,rows,N,K", [
    (FORWARD, 1, MOST, 4097, 8), (DX, 1, MOST, 8, 4097), (I8, 1, MOST, 4097, 8),  # 2^25 x 65 tiles
    (FORWARD, 1, MOST + 1, 8, 8), (DW, 1, MOST + 1, 8, 8),
    (DW, 4097, 8, 8, 8), (FORWARD, 1, 8, (1 << 20) + 1, 8), (DW, 1, 8, 8, (1 << 20) + 1),
    (FORWARD, 1, 8, 1 << 16, 1 << 15), (DW, 1, 8, 1 << 16, 1 << 15), (I8, 1, 8, 1 << 16, 1 << 16),  # 4 GiB a group
])
def test_sizes_outside_the_limits(op, G, rows, N, K):
    with pytest.raises(moe.MoeError):
        moe.moe_matmul_workspace_size(op, moe.MOE_BF16, G, rows, N, K)


@pytest.mark.parametrize("rows,status", [((1 << 23) + 1, moe.MOE_ERR_INVALID_ARG), (MOST, moe.MOE_ERR_INVALID_ARG),
                                         (MOST + 1, moe.MOE_ERR_UNSUPPORTED)])
def test_rows_of_the_quantizer(rows, status):
    """Accepted row counts get as far as the misaligned scales."""
    assert moe.load_library().moe_quantize_rows(moe.MOE_BF16, rows, 8, 0, FAKE, FAKE, ODD, None) == status
    assert ("scales" in moe.moe_last_error()) == (status == moe.MOE_ERR_INVALID_ARG)


@pytest.mark.parametrize("shape", [(), (0,), (2, 3)])
def test_shapes_of_the_offsets(shape):
    """The weight gradient takes its number of groups from the offsets: other shapes raise the binding's ValueError."""
    import torch

    t = torch.zeros((4, 8))
    with pytest.raises(ValueError, match="group_offsets"):
        moe.moe_grouped_matmul_dw(t, t, torch.zeros(shape, dtype=torch.int32))


@pytest.mark.parametrize("dtype,G,rows,N,K", [
    (moe.MOE_BF16, 3, 48782, 264, 602), (moe.MOE_F32, 1, 5469, 152, 552), (moe.MOE_F32, 14, 222560, 28, 1087)])
def test_ranges_of_the_weight_gradient_fill_the_chip(dtype, G, rows, N, K, tile=64, slots=768):
    """Where groups leave work-groups idle, their ranges (two partial sums of N x K each in the workspace) take two
    thirds of them or more, of three 64 x 64 tiles to a CU."""
    n = moe.moe_matmul_workspace_size(DW, dtype, G, rows, N, K)
    ranges = n // (2 * N * K * 4)
    tiles = -(-N // tile) * -(-K // tile)
    assert 2 / 3 * slots <= ranges * tiles <= slots * 1.05
