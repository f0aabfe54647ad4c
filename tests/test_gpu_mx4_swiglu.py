"""SwiGLU before the microscaled 4-bit codes: the same value that the rest of the library computes, over every finite gate."""
import numpy as np
import pytest

import moe_layer_forward_amd as moe

pytestmark = pytest.mark.gpu
N = 128  # values of a row


def _torch():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def _library_swiglu(x):
    """SiLU(gate) * up in fp32 as the layer's experts compute it: weights that pick single values, whose sums with zeros are
    exact."""
    torch = _torch()
    cfg = moe.make_config(2 * N, N, 1, 1, n_shared_experts=0, dtype=moe.MOE_F32)
    eye = torch.eye(2 * N, device="cuda")
    gate, up, down = eye[:N].contiguous(), eye[N:].contiguous(), eye[:, :N].contiguous()
    offsets = torch.tensor([0, len(x)], dtype=torch.int32, device="cuda")
    return moe.moe_grouped_swiglu(cfg, offsets, len(x), x, gate[None], up[None], down[None])[:, :N].contiguous()


@pytest.mark.parametrize("low,high", [(-8.0, 8.0), (-90.0, -86.0), (-100.0, 100.0)])
def test_codes_are_those_of_the_library_s_swiglu(low, high):
    """Random gates, and factors that bring every second product next to a tie of its code or to a power of two: within a few
    units of fp32, where any other value than that of swiglu_f32 would get another code somewhere."""
    torch = _torch()
    rng = np.random.default_rng(int(high - low))
    g = rng.uniform(low, high, (512, N)).astype(np.float32).astype(np.float64)
    silu = g / (1 + np.exp(-g))
    to = rng.choice([1.25, 1.75, 2.5, 3.5, 5.0, 4.0, 7.9999995], g.shape) * (1 + rng.integers(-9, 10, g.shape) * 2.0 ** -24)
    u = np.where(np.arange(N) % 2 == 1, to / np.where(silu == 0, 1, silu), rng.standard_normal(g.shape) * 3)
    x = torch.from_numpy(np.concatenate([g, np.clip(u, -3e38, 3e38)], axis=1)).float().cuda()
    v = _library_swiglu(x)
    codes, scales = moe.moe_quantize_mx4(x, swiglu=True)
    want_codes, want_scales = moe.moe_quantize_mx4(v)
    assert torch.equal(scales, want_scales)
    # the sums of _library_swiglu lose the sign of a zero (-0 + 0 = +0), which the codes keep: there magnitudes only
    pairs = (v == 0).view(len(v), -1, 2)
    keep = 0xff - 0x08 * pairs[..., 0].int() - 0x80 * pairs[..., 1].int()
    assert torch.equal(codes & keep, want_codes & keep), int((codes & keep != want_codes & keep).sum())


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_the_largest_gates_are_finite(dt):
    """SiLU(g) = g from some 20 on, up to the type's largest value: no block becomes NaN while g u is finite."""
    torch = _torch()
    t = getattr(torch, dt)
    top = torch.finfo(t).max
    gates = torch.tensor([1e30, 1e38, 2.3e38, 2.36e38, 2.5e38, 3e38, 3.3e38, top, -1e30, -2.36e38, -3e38, -top], dtype=t)
    for factor in (2.0 ** -100, -(2.0 ** -3), 1.0):
        x = torch.zeros((len(gates), 64), dtype=t)
        x[:, 5], x[:, 37] = gates, factor
        codes, scales = moe.moe_quantize_mx4(x.cuda(), swiglu=True)
        v = torch.zeros((len(gates), 32))
        v[:, 5] = torch.where(gates > 0, gates.float() * factor, torch.zeros(len(gates)))
        want_codes, want_scales = moe.moe_quantize_mx4(v.cuda())
        assert torch.equal(scales, want_scales) and int(scales.max()) < 255
        assert torch.equal(codes & 0x77, want_codes & 0x77) and torch.equal(codes[:8], want_codes[:8])
