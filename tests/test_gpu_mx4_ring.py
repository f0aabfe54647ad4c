"""The stream of weights for groups of few rows where an item is one window: every step changes the item."""
import ctypes

import pytest
from test_gpu_mx4 import _exact_product, _offsets

import moe_layer_forward_amd as moe

pytestmark = pytest.mark.gpu
SIZES = [3, 0, 12, 1, 1, 7] * 40


@pytest.mark.parametrize("N,K", [(900, 32), (900, 96), (1000, 256), (641, 480), (900, 512), (385, 1024)])
@pytest.mark.parametrize("index_rows", [0, 50])
def test_items_of_one_window(N, K, index_rows):
    _exact_product(SIZES, N, K, index_rows)


def test_items_of_one_window_of_more_groups_than_are_sorted():
    _exact_product([1] * 300 + [0] * 300 + [30] * 100, 520, 512, 0)


def test_these_sizes_run_on_the_ring():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    hip, events = ctypes.CDLL("libamdhip64.so"), (ctypes.c_void_p * 8)()
    for i in range(8):
        e = ctypes.c_void_p()
        assert hip.hipEventCreate(ctypes.byref(e)) == 0
        events[i] = e
    b = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    G, rows = len(SIZES), sum(SIZES)
    try:
        for N, K in ((900, 32), (641, 480), (385, 1024)):
            args = b(rows, K // 2), b(rows, moe.mx4_scale_cols(K)), b(G, N, K // 2), b(G, N, moe.mx4_scale_cols(K))
            moe.moe_profile_events(events, 8)
            moe.moe_matmul_mx4(*args, _offsets(SIZES))
            torch.cuda.synchronize()
            assert [moe.moe_profile_kernel(i) for i in range(moe.moe_profile_count())] == ["matmul_mx4_ring"], (N, K)
    finally:
        moe.moe_profile_events(None, 0)
