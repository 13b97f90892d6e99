/*
 * moe_layer.h -- C ABI of the whole mixture-of-experts layer for a few tokens (a decode step), for
 * GB300 (sm_103a).
 *
 *   logits[t, e] = sum_h x[t, h] w_router[e, h]                         (float32)
 *   the experts of token t and their weights: the gating op of mrr_gating.h on logits (its
 *   normalisation, bias, groups, top-k and scaling), weights kept in float32
 *   h[t, e, i]   = silu(sum_h x[t, h] w13[e, i, h]) * sum_h x[t, h] w13[e, I + i, h]
 *   y[t, n]      = sum over token t's experts of weight * sum_i h[t, e, i] w2[e, n, i]
 *
 * Sums are held in float32.  y is rounded once to x's type.  Between the two products weight * h goes
 * on as the sum of two 16-bit values (x's type, float16 for MXFP4 weights; float16 with a power of two
 * for each 16 elements), whose error does not show in y.  With MXFP4 weights, bfloat16 x and more than 4
 * tokens it is one float16 value: 2^-12, beside y's own rounding of 2^-9.
 *
 * Conventions are those of mrr_v2.h.
 */
#ifndef MOE_LAYER_H
#define MOE_LAYER_H

#include "moe_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* most tokens moe_few_token_layer_run takes; more go through the re-routing op and the grouped product where the
 * weights are MXFP4 (there is no grouped product of 16-bit weights) */
#define MOE_LAYER_MAX_TOKENS 64

/* Workspace bytes of moe_few_token_layer_run (host only); 0 where a size is out of range. */
size_t moe_few_token_layer_workspace(int64_t T, int64_t H, int64_t E, int64_t I, int64_t k);

/*
 * moe_few_token_layer_run -- enqueue the layer on `stream`.
 *   x            [T, H] in dt (MOE_F16 or MOE_BF16)                                      (read)
 *   w_router     [E, H] in dt; bias [E] in dt or NULL                                    (read)
 *   w13, w2      [E, 2 I, H] (I gate rows, then I up rows) and [E, H, I], both in w_dt: x's type
 *                (scales NULL) or MOE_MXFP4 with w13_scales, w2_scales                   (read)
 *   k, k_group, group_count, routed_scaling_factor, eps, group_select_mode, norm_type: as in
 *                mrr_gating_topk_run
 *   y            [T, H] in dt                                                            (written)
 *   topk_weight, expert_idx   [T, k] float32 and int32, or NULL                          (written)
 *   workspace    >= moe_few_token_layer_workspace(...) bytes, 256-byte aligned; its contents need
 *                not be initialised; status with mrr_v2_read_status (MRR_ERR_TIMEOUT: a bounded
 *                wait gave up, the outputs are unspecified)
 * Every expert index is in range whatever the logits hold; a token with a NaN logit gets
 * unspecified experts.  A NaN or infinity in x reaches that token's outputs only, and one in an expert's weights
 * those of the tokens that chose it.  The same inputs give the same bits; a token's last bits may differ with the
 * tokens beside it, as how sums are shared out depends on how many experts all of them reach.
 * Host errors: MRR_ERR_DTYPE, MRR_ERR_ATTR, MRR_ERR_SHAPE (T outside 0 .. MOE_LAYER_MAX_TOKENS, H
 * or I outside 1 .. 65536 or, with MXFP4 weights, odd; E outside 1 .. 1024; k outside 1 .. min(E,
 * 64); grouping as in mrr_gating_topk_run), MRR_ERR_NULL, MRR_ERR_ALIGN (a pointer not aligned to
 * its type), MRR_ERR_WORKSPACE, MRR_ERR_CUDA.
 */
mrr_status moe_few_token_layer_run(const void *x, moe_dtype dt, int64_t T, int64_t H, const void *w_router, int64_t E,
                                   const void *bias, const void *w13, const uint8_t *w13_scales, const void *w2,
                                   const uint8_t *w2_scales, moe_dtype w_dt, int64_t I, int64_t k, int64_t k_group,
                                   int64_t group_count, float routed_scaling_factor, float eps,
                                   int64_t group_select_mode, int64_t norm_type, void *y, float *topk_weight,
                                   int32_t *expert_idx, void *workspace, size_t workspace_bytes, mrr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LAYER_H */
