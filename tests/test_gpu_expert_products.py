"""The grouped products used together, as examples/expert_products.py does: a training step's gradients through an
expert layer against float64, training that learns, and the 8-bit experts against the bf16 ones."""
import os
import sys

import numpy as np
import pytest

import moe_layer_forward_amd as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


def _example():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import expert_products
    finally:
        sys.path.pop(0)
    return torch, expert_products


@pytest.mark.parametrize("T,H,inner,E,K", [(50, 128, 128, 6, 2), (200, 384, 256, 5, 3)])
def test_layer_gradients_against_float64(T, H, inner, E, K):
    """fp32 experts: every sum has at most max(2 I, H, T K) terms; with normal data the gradients' relative 2-norm
    error is far below that length's worst case, (depth + 16) 2^-23."""
    torch, ex = _example()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    cfg = moe.make_config(hidden_size=H, moe_intermediate_size=inner, n_routed_experts=E, top_k=K, n_shared_experts=0,
                          dtype="f32")

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    x = normal(T, H).requires_grad_()
    gu = normal(E, 2 * inner, H, scale=H ** -0.5).requires_grad_()
    dn = normal(E, H, inner, scale=inner ** -0.5).requires_grad_()
    dy = normal(T, H)
    weights, offsets, row_token, pair_row = ex.dispatch(cfg, x.detach(), normal(E, H, scale=0.1))
    y = ex.experts(cfg, x, gu, dn, (weights, offsets, row_token, pair_row))
    (y * dy).sum().backward()

    x6, gu6, dn6 = (t.detach().double().cpu().requires_grad_() for t in (x, gu, dn))
    off, tok = offsets.cpu().numpy(), row_token.cpu().long()
    rows = torch.zeros((T * K, H), dtype=torch.float64)
    parts = []
    for e in range(E):
        a = x6[tok[off[e]:off[e + 1]]]
        g, u = (a @ gu6[e].T).chunk(2, dim=1)
        parts.append((g * torch.sigmoid(g) * u) @ dn6[e].T)
    rows = torch.cat(parts)
    ref = (rows[pair_row.cpu().long()] * weights.double().cpu()[:, :, None]).sum(dim=1)
    (ref * dy.double().cpu()).sum().backward()
    bound = (max(2 * inner, H, T * K) + 16) * 2.0 ** -23
    for name, got, want in (("y", y, ref), ("dx", x.grad, x6.grad), ("d gate_up", gu.grad, gu6.grad),
                            ("d down", dn.grad, dn6.grad)):
        a, b = got.detach().double().cpu().numpy(), want.detach().numpy()
        err = np.linalg.norm(a - b) / np.linalg.norm(b)
        print(f"{name}: relative error {err:.2e} (bound {bound:.2e})", flush=True)
        assert err <= bound, name


def test_example_learns_and_serves_in_8_bits():
    """The loss falls to less than half; an 8-bit operand is off by about max / 127 / sqrt(12) of its rms, 0.7% for
    normal rows (max about 3 rms), so two products of two such operands stay within 3%."""
    _, ex = _example()
    first, last, error = ex.main()
    assert last < 0.5 * first
    assert error < 0.03
