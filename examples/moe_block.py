"""One mixture-of-experts block, as a serving rank runs it, on MXFP4 expert weights.

Prefill: the norm with its rows in MXFP4, the routing decision, rows laid out as an expert-parallel
exchange delivers them (one segment per source rank and expert), re-routed to expert-major order, the
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


def delivered(codes, scales, expert, weight, E, ranks):
    """What an exchange delivers: rank by rank, each rank's rows in expert order, with the row of each of their slots."""
    T, k = expert.shape
    rank = (torch.arange(T, device=codes.device) * ranks // T).int()
    at_once, parts, ahead = 4096 // E, [], 0     # the experts of one sort are 4096 or fewer: a few ranks' at a time
    for r in range(0, ranks, at_once):
        n = min(at_once, ranks - r)
        to = -(-(r + n) * T // ranks)            # the first token of rank r + n
        t = slice(ahead, to)
        rows, row_scales, _, row_idx, counts, row_weight = moe.moe_sort_tokens(
            codes[t], expert[t] + E * (rank[t] - r)[:, None], n * E, per_token_scales=scales[t],
            expert_topk_weight=weight[t])
        parts.append((rows, row_scales, row_idx + k * ahead if ahead else row_idx, counts.view(n, E), row_weight))
        ahead = to
    return parts[0] if len(parts) == 1 else [torch.cat(p) for p in zip(*parts)]


def prefill(x, w, k, ranks, quantised=None):
    """The block on x [T, H] bfloat16, as if `ranks` source ranks had each sent a share of the tokens.
    `quantised`: x's MXFP4 rows and scales, where the norm in front has made them already.
    Every (rank, expert) pair needs a row, as the re-routing op asks."""
    T, H = x.shape
    E = w["router"].shape[0]
    weight, expert, _ = moe.moe_gating_top_k(x @ w["router"].t(), k, bias=w["bias"], **ROUTING)

    codes, scales = moe.moe_mx_quantize(x) if quantised is None else quantised
    rows, row_scales, row_idx, counts, row_weight = delivered(codes, scales, expert, weight, E, ranks)

    # expert-major, through the experts, and back
    rows, row_scales, _, num, row_weight = moe.moe_re_routing(
        rows, counts, per_token_scales=row_scales, expert_topk_weight=row_weight, tokens_dtype="float4_e2m1",
        check_status=True)
    h, h_scales = moe.moe_mx_grouped_matmul(rows, row_scales, num, w["w13"], w["s13"], gated=True, out_dtype="mxfp4")
    y = moe.moe_mx_grouped_matmul(h, h_scales, num, w["w2"], w["s2"], row_weight=row_weight, check_status=True)
    y, _, _ = moe.moe_re_routing_inverse(y, counts, check_status=True)
    return moe.moe_combine_tokens(y, row_idx)      # the weights are in y already


def normed_prefill(x, residual, gain, w, k, ranks):
    """The block with the residual's addition and the norm in front: (the block's result, the new residual)."""
    y, h, codes, scales = moe.moe_add_rms_norm(x, gain, residual, quant="mxfp4")
    return prefill(y, w, k, ranks, (codes, scales)), h


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
    gain = torch.ones(2048, dtype=torch.bfloat16, device="cuda")
    y, _ = normed_prefill(x, torch.zeros_like(x), gain, w, k=4, ranks=4)
    x = moe.moe_add_rms_norm(x[:8].contiguous(), gain)[0]
    z = decode(x, w, k=4)
    off = (y[:8].float() - z.float()).norm() / z.float().norm()
    print(f"prefill {tuple(y.shape)}, decode {tuple(z.shape)}: the first 8 tokens differ by {off:.3f} "
          "(prefill's activations are quantised to MXFP4, decode's are not)")


if __name__ == "__main__":
    main()
