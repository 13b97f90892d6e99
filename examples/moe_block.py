"""One mixture-of-experts block, as a serving rank runs it, on MXFP4 expert weights.

Prefill: the routing decision, rows quantised to MXFP4, laid out as an expert-parallel exchange
delivers them (one segment per source rank and expert), re-routed to expert-major order, the
experts' two products, the inverse move, and each token's weighted sum.  Decode: the whole layer in
one launch for a few tokens, with the same weights.

    python examples/moe_block.py        (from the repository root)
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import moe_expert_token_gb300 as moe  # noqa: E402

ROUTING = dict(k_group=2, group_count=4, group_select_mode=1, norm_type=1, routed_scaling_factor=2.5)


def weights(E, H, I, generator):
    """Router weights, bias and MXFP4 expert weights of a random layer."""
    rnd = lambda *s: torch.randn(*s, generator=generator, device="cuda")  # noqa: E731
    w = {"router": (rnd(E, H) * H ** -0.5).bfloat16(), "bias": (0.1 * rnd(E)).bfloat16()}
    w["w13"], w["s13"] = moe.moe_mx_quantize(rnd(E, 2 * I, H) * H ** -0.5)
    w["w2"], w["s2"] = moe.moe_mx_quantize(rnd(E, H, I) * I ** -0.5)
    return w


def prefill(x, w, k, ranks):
    """The block on x [T, H] bfloat16, as if `ranks` source ranks had each sent a share of the tokens.
    Every (rank, expert) pair needs a row, as the re-routing op asks."""
    T, H = x.shape
    E = w["router"].shape[0]
    weight, expert, _ = moe.moe_gating_top_k(x @ w["router"].t(), k, bias=w["bias"], **ROUTING)

    # what an exchange delivers: rank by rank, each rank's rows in expert order
    token = torch.arange(T, device=x.device).repeat_interleave(k)
    rank = token * ranks // T
    expert, weight = expert.flatten().long(), weight.flatten()
    order = torch.argsort(rank * E + expert, stable=True)
    counts = torch.bincount(rank * E + expert, minlength=ranks * E).view(ranks, E).int()
    codes, scales = moe.moe_mx_quantize(x)
    rows, row_scales = codes[token[order]], scales[token[order]]
    row_weight = weight[order].float().view(-1, 1)

    # expert-major, through the experts, and back
    rows, row_scales, _, num, row_weight = moe.moe_re_routing(
        rows, counts, per_token_scales=row_scales, expert_topk_weight=row_weight, tokens_dtype="float4_e2m1",
        check_status=True)
    h, h_scales = moe.moe_mx_grouped_matmul(rows, row_scales, num, w["w13"], w["s13"], gated=True, out_dtype="mxfp4")
    y = moe.moe_mx_grouped_matmul(h, h_scales, num, w["w2"], w["s2"], row_weight=row_weight, check_status=True)
    y, _, _ = moe.moe_re_routing_inverse(y, counts, check_status=True)
    return torch.zeros(T, H, device=x.device).index_add_(0, token[order], y.float()).to(x.dtype)


def decode(x, w, k):
    """The block on a few tokens x [T <= 64, H]."""
    return moe.moe_few_token_layer(x, w["router"], w["w13"], w["w2"], k, bias=w["bias"], w13_scales=w["s13"],
                                   w2_scales=w["s2"], check_status=True, **ROUTING)


def main():
    from moe_expert_token_gb300 import build

    build.build()
    generator = torch.Generator(device="cuda").manual_seed(0)
    w = weights(E=32, H=2048, I=1024, generator=generator)
    x = torch.randn(4096, 2048, generator=generator, device="cuda").bfloat16()
    y = prefill(x, w, k=4, ranks=4)
    z = decode(x[:8].contiguous(), w, k=4)
    off = (y[:8].float() - z.float()).norm() / z.float().norm()
    print(f"prefill {tuple(y.shape)}, decode {tuple(z.shape)}: the first 8 tokens differ by {off:.3f} "
          "(prefill's activations are quantised to MXFP4, decode's are not)")


if __name__ == "__main__":
    main()
