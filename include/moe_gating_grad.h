/*
 * moe_gating_grad.h -- C ABI of the gradient of the gating top-k op (mrr_gating.h), for GB300 (sm_103a).
 *
 * Conventions are those of mrr_v2.h.  The same inputs give the same bits.  Calls that may run at the same time need
 * workspaces of their own.  Calls may be captured in a CUDA graph.
 */
#ifndef MOE_GATING_GRAD_H
#define MOE_GATING_GRAD_H

#include "mrr_gating.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Workspace bytes of moe_gating_topk_grad_run (host only); 0 where a size is out of range. */
size_t moe_gating_topk_grad_workspace(int64_t T, int64_t e);

/*
 * moe_gating_topk_grad_run -- the gradient of mrr_gating_topk_run's y_out and norm_out, for the experts it chose.
 *   With s = norm(x) + the row's bias, p_j = s[expert_idx_j], P = sum_j p_j + eps, c = routed_scaling_factor:
 *     ds = grad_norm_out, and at expert_idx_j  + c / P * (grad_y_j - sum_i grad_y_i p_i / P)
 *     softmax: grad_x = n (ds - sum_e ds n), n = softmax(x); sigmoid: grad_x = ds n (1 - n); softplus:
 *     grad_x = ds sigmoid(x)
 *     grad_bias = sum of ds over the rows that use bias, grad_additional_bias over those that do not
 *   All in float32, each rounded once; the choice of experts itself has no gradient.
 *   grad_y [T, k] in dt; x [T, e] in dt; expert_idx [T, k] int32 (an entry outside 0 .. e - 1 counts
 *   as no expert); bias, additional_bias, additional_token_mask as mrr_gating_topk_run had them;
 *   grad_norm_out [T, e] float32 or NULL                                                  (read)
 *   grad_x [T, e] in dt; grad_bias, grad_additional_bias [e] in dt, or NULL               (written)
 *   workspace  >= moe_gating_topk_grad_workspace(T, e) bytes, 256-byte aligned, where a bias gradient is asked for;
 *              not initialised
 * Host errors: MRR_ERR_DTYPE, MRR_ERR_ATTR (norm_type), MRR_ERR_SHAPE (T < 0 or above 2^31 - 1, e outside 1 .. 1024,
 * k outside 1 .. min(e, 64)), MRR_ERR_NULL, MRR_ERR_ALIGN (a pointer not aligned to its type), MRR_ERR_WORKSPACE,
 * MRR_ERR_CUDA.
 */
mrr_status moe_gating_topk_grad_run(const void *grad_y, const void *x, mrr_gate_dtype dt, int64_t T, int64_t e,
                                    int64_t k, const int32_t *expert_idx, const void *bias,
                                    const void *additional_bias, const uint8_t *additional_token_mask,
                                    const float *grad_norm_out, float routed_scaling_factor, float eps,
                                    int64_t norm_type, void *grad_x, void *grad_bias, void *grad_additional_bias,
                                    void *workspace, size_t workspace_bytes, mrr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GATING_GRAD_H */
