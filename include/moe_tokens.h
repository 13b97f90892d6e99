/*
 * moe_tokens.h -- C ABI of the moves between token order and expert order on one rank, for GB300
 * (sm_103a): tokens laid out by the experts that were chosen for them (what a rank sends into the
 * expert-parallel exchange, or hands to its own experts), the experts' rows back to their tokens,
 * weighted and summed, and the gradients of both.
 *
 *   slot       i = t * k + j: the j-th expert of token t; T * k slots
 *   key(i)     expert_idx[i] - first_expert where that is one of 0 .. E - 1 (an expert held here);
 *              another value, as -1 in a padded token, gives the slot no row
 *   rows       in order of (key, i): expert 0's slots in slot order, then expert 1's, and so on;
 *              behind them, in slot order, one row of zeros for each slot without a row
 *   row_idx    [T, k] int32: a slot's row, -1 where it has none
 *   token_idx  [T * k] int32: a row's slot, -1 for the rows of zeros
 *
 * Conventions are those of mrr_v2.h: device pointers unless stated otherwise, buffers owned by
 * the caller, nothing allocated, work only enqueued on `stream` (the current device), errors
 * found on the host returned at once with nothing enqueued; inputs and outputs do not overlap.
 * The same inputs give the same bits (of grad_weight, for the same T).  Calls that may run at the same time
 * need workspaces of their own.  Calls may be captured in a CUDA graph.
 */
#ifndef MOE_TOKENS_H
#define MOE_TOKENS_H

#include "moe_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* most experts a token has, and most experts held here */
#define MOE_SORT_MAX_K 64
#define MOE_SORT_MAX_EXPERTS 4096

/* Workspace bytes of moe_sort_run (host only); 0 where none is needed or a size is out of range. */
size_t moe_sort_workspace(int64_t T, int64_t k, int64_t E);

/*
 * moe_sort_run -- lay out the rows of T tokens by expert.
 *   expert_idx      [T, k] int32 or int64 (idx_is_i64)                                    (read)
 *   first_expert, E the experts held here: first_expert .. first_expert + E - 1
 *   x               T rows of row_bytes bytes, row t at x + t * row_stride; NULL (row_bytes 0) to
 *                   make the indices only                                                 (read)
 *   scales          [T] rows of scale_row_bytes bytes without gaps, or NULL               (read)
 *   weight          [T, k] in weight_dt (F16, BF16, F32), or NULL                         (read)
 *   sorted_x        [T * k] rows of row_bytes bytes                                       (written)
 *   sorted_scales   [T * k] rows of scale_row_bytes bytes; NULL without scales            (written)
 *   sorted_weight   [T * k] float32; NULL without weights                                 (written)
 *   token_idx, row_idx  as above                                                          (written)
 *   expert_num      [E] in expert_idx's type: each expert's rows (expert_num_type 1) or their
 *                   inclusive prefix (0), as the re-routing op writes them                (written)
 *   workspace       >= moe_sort_workspace(T, k, E) bytes, 256-byte aligned (NULL where that is 0);
 *                   its contents need not be initialised
 * Rows, scales and weights of zeros (all bytes 0) fill what is behind the last expert's rows.
 * Host errors: MRR_ERR_DTYPE, MRR_ERR_ATTR (expert_num_type), MRR_ERR_SHAPE (T < 0, k outside 1 ..
 * 64, E outside 1 .. 4096, first_expert + E - 1 above 2^63 - 1, T * k above 2^31 - 1, row_bytes outside
 * 0 .. 2^24, row_stride < row_bytes, scale_row_bytes outside 1 .. 2^20 with scales), MRR_ERR_NULL, MRR_ERR_ALIGN (expert_idx, weight or
 * a written index not aligned to its type), MRR_ERR_WORKSPACE, MRR_ERR_CUDA.
 */
mrr_status moe_sort_run(const void *expert_idx, int idx_is_i64, int64_t T, int64_t k, int64_t first_expert, int64_t E,
                        const void *x, int64_t row_bytes, int64_t row_stride, const void *scales,
                        int64_t scale_row_bytes, const void *weight, moe_dtype weight_dt, void *sorted_x,
                        void *sorted_scales, float *sorted_weight, int32_t *token_idx, int32_t *row_idx,
                        void *expert_num, int64_t expert_num_type, void *workspace, size_t workspace_bytes,
                        mrr_stream_t stream);

/*
 * moe_combine_run -- y[t] = sum over j of weight[t, j] * rows[row_idx[t, j]], float32 sums in the
 *   order of j, rounded once; without weights each counts once (the gradient of moe_sort_run: rows
 *   then are the gradient of sorted_x).  A slot whose row_idx is outside 0 .. R - 1 adds nothing,
 *   and its weight is not used; a token without any row is zero.  (T k tokens of one slot each, rows of one element: the
 *   gradient of moe_sort_run's weights, rows then being the gradient of sorted_weight.)
 *   rows [R, H] in dt (read), row_idx [T, k] int32 (read), weight [T, k] in weight_dt or NULL (read),
 *   y [T, H] in dt (written).
 * Host errors: MRR_ERR_DTYPE, MRR_ERR_SHAPE (T, R < 0 or above 2^31 - 1, T + R / 32 above 2^31 - 2434, H outside
 * 1 .. 2^20, k outside 1 .. 64), MRR_ERR_NULL, MRR_ERR_ALIGN, MRR_ERR_CUDA.
 */
mrr_status moe_combine_run(const void *rows, moe_dtype dt, int64_t R, int64_t H, const int32_t *row_idx, int64_t T,
                           int64_t k, const void *weight, moe_dtype weight_dt, void *y, mrr_stream_t stream);

/*
 * moe_combine_grad_run -- the gradient of moe_combine_run:
 *   grad_rows[row_idx[t, j]] = weight[t, j] * grad_y[t]; a row whose token_idx is negative: zeros
 *   grad_weight[t, j] = sum over h of grad_y[t, h] * rows[row_idx[t, j], h], in float32, rounded
 *                       once; 0 for a slot without a row
 *   grad_y [T, H] in dt, rows [R, H] in dt (NULL with grad_weight NULL), row_idx [T, k], token_idx
 *   [R], both of one moe_sort_run: every row is some slot's, or has a negative token_idx  (read)
 *   grad_rows [R, H] in dt, grad_weight [T, k] in weight_dt or NULL                       (written)
 * Errors as for moe_combine_run; grad_weight needs weight.
 */
mrr_status moe_combine_grad_run(const void *grad_y, const void *rows, moe_dtype dt, int64_t R, int64_t H,
                                const int32_t *row_idx, const int32_t *token_idx, int64_t T, int64_t k,
                                const void *weight, moe_dtype weight_dt, void *grad_rows, void *grad_weight,
                                mrr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TOKENS_H */
