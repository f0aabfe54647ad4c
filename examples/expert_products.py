"""An MoE layer's experts trained with the grouped products, then served from 8-bit integers.

    python examples/expert_products.py

The layer is the library's (sigmoid router, top-K, SwiGLU experts, weighted combine), with the experts as plain
tensors: ``moe_grouped_matmul`` is differentiable by itself; ``GroupedProduct`` is the same node written out with
``moe_grouped_matmul_dx`` and ``moe_grouped_matmul_dw``, where the routing knows each token's rows and ``moe_combine``
adds their gradients in one pass.  ``int8_experts`` runs the trained experts through ``moe_quantize_rows`` and
``moe_matmul_i8``.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_layer_forward_amd as moe  # noqa: E402


class GroupedProduct(torch.autograd.Function):
    """y[r] = W[g(r)] x[row_index[r]] (or x[r]), with gradients for x and W.

    pair_row [T, K] names the rows of each token where rows are gathered: a token's gradient is the sum over
    them, which moe_combine adds with weights 1."""

    @staticmethod
    def forward(ctx, x, w, offsets, row_index=None, pair_row=None, cfg=None):
        ctx.save_for_backward(x, w)
        ctx.route = offsets, row_index, pair_row, cfg
        return moe.moe_grouped_matmul(x, w, offsets, row_index=row_index)

    @staticmethod
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        offsets, row_index, pair_row, cfg = ctx.route
        dy = dy.contiguous()
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = moe.moe_grouped_matmul_dx(dy, w, offsets)
            if row_index is not None:
                dx = moe.moe_combine(cfg, dx, pair_row, torch.ones(pair_row.shape, device=dy.device))
        if ctx.needs_input_grad[1]:
            dw = moe.moe_grouped_matmul_dw(dy, x, offsets, row_index=row_index)
        return dx, dw, None, None, None, None


def dispatch(cfg, x, w_router):
    """(weights [T, K], offsets [E + 1], row_token [T K], pair_row [T, K]) of the layer's routing."""
    ids, weights = moe.moe_route(cfg, x, w_router)
    offsets, row_token, pair_row, _ = moe.moe_permute(cfg, ids)
    return weights, offsets, row_token, pair_row


def experts(cfg, x, w_gate_up, w_down, routing):
    """The routed experts in the type of x: gate and up side by side [E, 2 I, H], down [E, H, I]."""
    weights, offsets, row_token, pair_row = routing
    gate_up = GroupedProduct.apply(x, w_gate_up, offsets, row_token, pair_row, cfg)
    gate, up = gate_up.float().chunk(2, dim=1)
    h = (torch.nn.functional.silu(gate) * up).to(x.dtype)
    y_rows = GroupedProduct.apply(h, w_down, offsets)
    return (y_rows[pair_row.long()].float() * weights[:, :, None]).sum(dim=1)


def to_int8(w):
    """A weight [E, N, K] as codes and one scale per output channel (a channel is a row of N x K)."""
    codes, scales = moe.moe_quantize_rows(w.reshape(-1, w.shape[-1]))
    return codes.view(w.shape), scales.view(w.shape[:-1])


def int8_experts(cfg, x, gate_up8, down8, routing):
    """The routed experts in 8-bit integers: two quantizations, two products, the combine."""
    weights, offsets, row_token, pair_row = routing
    q, s = moe.moe_quantize_rows(x)
    gate_up = moe.moe_matmul_i8(q, s, *gate_up8, offsets, row_index=row_token, y_dtype=moe.MOE_F32)
    h, sh = moe.moe_quantize_rows(gate_up, swiglu=True)
    y_rows = moe.moe_matmul_i8(h, sh, *down8, offsets)
    return moe.moe_combine(cfg, y_rows, pair_row, weights)


def main(T=256, H=256, inner=128, E=8, K=2, steps=30, lr=0.02, seed=0):
    """Trains the experts towards a teacher of the same shape; returns (first loss, last loss, relative error of
    the 8-bit layer against the trained one)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(scale).bfloat16()

    cfg = moe.make_config(hidden_size=H, moe_intermediate_size=inner, n_routed_experts=E, top_k=K, n_shared_experts=0)
    x = normal(T, H)
    routing = dispatch(cfg, x, normal(E, H, scale=0.1))
    with torch.no_grad():
        target = experts(cfg, x, normal(E, 2 * inner, H, scale=H ** -0.5), normal(E, H, inner, scale=inner ** -0.5), routing)
    # fp32 master weights, the products in bf16
    gate_up = normal(E, 2 * inner, H, scale=H ** -0.5).float().requires_grad_()
    down = normal(E, H, inner, scale=inner ** -0.5).float().requires_grad_()
    losses = []
    for step in range(steps):
        y = experts(cfg, x, gate_up.bfloat16(), down.bfloat16(), routing)
        loss = (y - target).square().mean()
        loss.backward()
        with torch.no_grad():
            for p in (gate_up, down):
                p -= lr * H * p.grad  # per token: the loss is a mean over H as well
                p.grad = None
        losses.append(float(loss.detach()))
        if step % 10 == 0 or step == steps - 1:
            print(f"step {step}: loss {losses[-1]:.4f}", flush=True)
    with torch.no_grad():
        y = experts(cfg, x, gate_up.bfloat16(), down.bfloat16(), routing)
        y8 = int8_experts(cfg, x, to_int8(gate_up.bfloat16()), to_int8(down.bfloat16()), routing).float()
        error = float((y8 - y).norm() / y.norm())
    print(f"8-bit experts against bf16: relative error {error:.4f}", flush=True)
    return losses[0], losses[-1], error


if __name__ == "__main__":
    main()
