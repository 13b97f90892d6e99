"""A mixture-of-experts block in training: the package's forward calls and their gradients as torch
functions, around experts that are torch's own matrix products.

    python examples/moe_training.py        (from the repository root)

norm -> router -> top-k -> tokens laid out by expert -> experts -> weighted sum, and all of it backwards.  A
backward pass that is captured in a CUDA graph calls the gradients themselves (moe.*_grad), as these
functions do.
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402
from torch.autograd.function import once_differentiable  # noqa: E402

import moe_expert_token_gb300 as moe  # noqa: E402


class AddRmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gain, eps):
        y, h, _, _ = moe.moe_add_rms_norm(x, gain, residual, eps=eps)
        ctx.save_for_backward(h, gain)
        ctx.eps = eps
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_h):
        h, gain = ctx.saved_tensors
        grad, grad_gain = moe.moe_add_rms_norm_grad(grad_y.contiguous(), h, gain, grad_h=grad_h.contiguous(), eps=ctx.eps)
        return grad, grad, grad_gain, None


class GatingTopK(torch.autograd.Function):
    """``routing``: moe_gating_top_k's other arguments, a mask among them; the biases, which have gradients, come by themselves."""

    @staticmethod
    def forward(ctx, logits, k, routing, bias=None, additional_bias=None):
        weight, expert, _ = moe.moe_gating_top_k(logits, k, bias=bias, additional_bias=additional_bias, **routing)
        ctx.save_for_backward(logits, expert, bias, additional_bias)
        ctx.kw = {n: routing[n] for n in ("additional_token_mask", "routed_scaling_factor", "eps", "norm_type") if n in routing}
        ctx.mark_non_differentiable(expert)
        return weight, expert

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_weight, _):
        logits, expert, bias, additional_bias = ctx.saved_tensors
        grad, grad_bias, grad_additional = moe.moe_gating_top_k_grad(grad_weight.contiguous(), logits, expert, bias=bias,
                                                                     additional_bias=additional_bias, **ctx.kw)
        return grad, None, None, grad_bias, grad_additional


class SortTokens(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, expert, num_experts):
        rows, _, token_idx, row_idx, num, _ = moe.moe_sort_tokens(x, expert, num_experts)
        ctx.save_for_backward(row_idx)
        ctx.mark_non_differentiable(token_idx, row_idx, num)
        return rows, token_idx, row_idx, num

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_rows, *_):
        return moe.moe_sort_tokens_grad(grad_rows.contiguous(), *ctx.saved_tensors), None, None


class CombineTokens(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, row_idx, token_idx, weight):
        ctx.save_for_backward(rows, row_idx, token_idx, weight)
        return moe.moe_combine_tokens(rows, row_idx, weight)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        grad_rows, grad_weight = moe.moe_combine_tokens_grad(grad_y.contiguous(), *ctx.saved_tensors)
        return grad_rows, None, None, grad_weight


ROUTING = dict(norm_type=1, routed_scaling_factor=2.5)


def parameters(E, H, I, generator, dtype=torch.bfloat16):
    """The router's, the norm's and the experts' weights of a random block."""
    rnd = lambda *s: torch.randn(*s, generator=generator, device="cuda")  # noqa: E731
    p = {"gain": 1 + 0.1 * rnd(H), "router": rnd(E, H) * H ** -0.5, "w13": rnd(E, 2 * I, H) * H ** -0.5,
         "w2": rnd(E, H, I) * I ** -0.5}
    return {n: v.to(dtype).requires_grad_() for n, v in p.items()}


def block(x, residual, p, k):
    """(the block's result, the new residual) for x and residual [T, H]."""
    E = p["router"].shape[0]
    y, h = AddRmsNorm.apply(x, residual, p["gain"], 1e-6)
    weight, expert = GatingTopK.apply(y @ p["router"].t(), k, ROUTING)
    rows, token_idx, row_idx, num = SortTokens.apply(y, expert, E)
    outs = []
    for e, r in enumerate(rows.split(num.tolist())):     # each expert's rows, one after the other
        g, u = (r @ p["w13"][e].t()).chunk(2, -1)
        outs.append((torch.nn.functional.silu(g) * u) @ p["w2"][e].t())
    return CombineTokens.apply(torch.cat(outs), row_idx, token_idx, weight), h


def main():
    from moe_expert_token_gb300 import build

    build.build()
    generator = torch.Generator(device="cuda").manual_seed(0)
    p = parameters(E=16, H=1024, I=512, generator=generator)
    optimizer = torch.optim.Adam(p.values(), lr=1e-3)    # (steps that bfloat16 weights of 0.03 can take)
    x = torch.randn(2048, 1024, generator=generator, device="cuda").bfloat16()
    target = torch.randn(2048, 1024, generator=generator, device="cuda").bfloat16()
    for step in range(3):
        y, h = block(x, torch.zeros_like(x), p, k=4)
        loss = (y + h - target).float().square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        print(f"step {step}: loss {loss.item():.4f}")


if __name__ == "__main__":
    main()
