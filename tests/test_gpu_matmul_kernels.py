"""The grouped products on each of their kernels: what a call launched is read from the library's own
profile (moe_profile_events), so that a test which is about one kernel fails where another runs."""
import ctypes

import numpy as np
import pytest

import moe_layer_forward_amd as moe

pytestmark = pytest.mark.gpu


def _torch():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def _launched(call, n_events=16):
    """(what call returns, [(kernel, ms)] of what it launched)."""
    torch = _torch()
    events = [torch.cuda.Event(enable_timing=True) for _ in range(n_events)]
    for e in events:
        e.record()  # torch creates an event when it is first recorded
    handles = (ctypes.c_void_p * n_events)(*[e.cuda_event for e in events])
    torch.cuda.synchronize()
    moe.moe_profile_events(handles, n_events)
    try:
        out = call()
        n = moe.moe_profile_count()
        names = [moe.moe_profile_kernel(i) for i in range(n)]
    finally:
        moe.moe_profile_events(None, 0)
    torch.cuda.synchronize()
    return out, [(k, events[2 * i].elapsed_time(events[2 * i + 1])) for i, k in enumerate(names)]


def test_profile_has_one_entry_per_launch():
    """A call whose sums are split launches the product and the join, and each is timed by itself."""
    torch = _torch()
    x = torch.randn((64, 8192), device="cuda").bfloat16()
    w = torch.randn((1, 128, 8192), device="cuda").bfloat16()
    dy = torch.randn((64, 128), device="cuda").bfloat16()
    rows = torch.randn((5000, 64), device="cuda")
    q, s = moe.moe_quantize_rows(x)
    qw, sw = moe.moe_quantize_rows(w[0])
    for call, want in (
            (lambda: moe.moe_grouped_matmul(x, w, None), ["matmul_tile128", "matmul_join"]),
            (lambda: moe.moe_grouped_matmul(x.float(), w.float(), None), ["matmul_any64", "matmul_join"]),
            (lambda: moe.moe_matmul_i8(q, s, qw[None], sw[None]), ["matmul_tile128", "matmul_join"]),
            (lambda: moe.moe_grouped_matmul_dw(rows, rows, None), ["matmul_any64", "matmul_join"]),
            (lambda: moe.moe_grouped_matmul_dx(dy, w, None), ["matmul_tile128"]),
            (lambda: moe.moe_quantize_rows(x), ["quantize_rows"])):
        _, got = _launched(call)
        assert [k for k, _ in got] == want
        assert all(ms > 0 for _, ms in got)
