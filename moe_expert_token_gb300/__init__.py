"""GB300-native MoE token re-routing (MoeReRoutingV2): rank-major -> expert-major.

The op lives in the CUDA library ``lib/libmrr_v2.so`` (C ABI: include/mrr_v2.h);
``moe_expert_token_gb300.mrr_v2`` is its ctypes binding and ``moe_re_routing`` the torch-level
call.  ``moe_expert_token_gb300.experts`` holds the operators on either side of it (include/moe_mx.h,
include/moe_layer.h): MXFP4 rows, the experts' products, and a whole layer for a few tokens.
``moe_expert_token_gb300.tokens`` holds what stands around the experts (include/moe_tokens.h,
include/moe_norm.h): the norm in front of them, tokens laid out by expert and back, and gradients.
Build the library with ``python -m moe_expert_token_gb300.build``.
"""
from .experts import (  # noqa: F401
    moe_few_token_layer,
    moe_few_token_layer_run,
    moe_few_token_layer_workspace,
    moe_mx_dequantize,
    moe_mx_dequantize_run,
    moe_mx_grouped_matmul,
    moe_mx_grouped_run,
    moe_mx_grouped_workspace,
    moe_mx_quantize,
    moe_mx_quantize_run,
)
from .mrr_v2 import (  # noqa: F401
    MrrError,
    load_library,
    moe_re_routing,
    moe_re_routing_inverse,
    moe_re_routing_multi,
    moe_re_routing_v1,
    moe_gating_top_k,
    mrr_gating_topk_run,
    mrr_v1_run,
    mrr_status_str,
    mrr_v2_plan,
    mrr_v2_read_status,
    mrr_v2_run,
    mrr_v2_run_multi,
    mrr_v2_run_plan,
    mrr_v2_run_plan_multi,
    mrr_v2_unroute,
    mrr_v2_unroute_plan,
)
from .tokens import (  # noqa: F401
    moe_add_rms_norm,
    moe_add_rms_norm_grad,
    moe_add_rms_norm_grad_run,
    moe_add_rms_norm_grad_workspace,
    moe_add_rms_norm_run,
    moe_combine_grad_run,
    moe_combine_run,
    moe_combine_tokens,
    moe_combine_tokens_grad,
    moe_dequantize_rows,
    moe_dequantize_rows_run,
    moe_gating_top_k_grad,
    moe_sort_run,
    moe_sort_tokens,
    moe_sort_tokens_grad,
    moe_sort_workspace,
    moe_gating_topk_grad_run,
    moe_gating_topk_grad_workspace,
)
