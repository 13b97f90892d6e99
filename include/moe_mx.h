/*
 * moe_mx.h -- C ABI of the MXFP4 operators around the re-routing op, for GB300 (sm_103a):
 * quantisation, its inverse, and the experts' products on expert-major rows.
 *
 * MXFP4 (OCP Microscaling Formats specification, version 1.0): a row of K elements is cut into
 * blocks of 32 (the last may be shorter).  A block has one e8m0 scale byte b, which stands for
 * 2^(b - 127) (255: NaN), and an element one e2m1 code: bit 3 is the sign, bits 0..2 the
 * magnitude 0, 0.5, 1, 1.5, 2, 3, 4, 6.  In memory, as the re-routing op moves them:
 *   codes   [rows, K/2] bytes; element 2i in the low four bits of byte i (MRR_F4E2M1 rows)
 *   scales  [rows, ceil(K/64), 2] bytes (MRR_SCALE_E8M0_AK2); where the last pair has no second
 *           block its byte is written as 127 and never used
 *
 * Conventions are those of mrr_v2.h: device pointers unless stated otherwise, buffers owned by
 * the caller, nothing allocated, work only enqueued on `stream` (the current device), errors
 * found on the host returned at once with nothing enqueued; inputs and outputs do not overlap.
 */
#ifndef MOE_MX_H
#define MOE_MX_H

#include "mrr_v2.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types of rows in memory; the first three agree with mrr_gate_dtype */
typedef enum moe_dtype {
    MOE_F16 = 0,
    MOE_BF16 = 1,
    MOE_F32 = 2,
    MOE_MXFP4 = 3    /* codes and scales as above */
} moe_dtype;

/*
 * moe_mx_quantize_run -- x [rows, K] in dt, row r at x + r * row_stride elements, to MXFP4.
 *   The block's scale is 2^(floor(log2 m) - 2), m its largest magnitude, the exponent held to
 *   -127 .. 127; an element is x / scale rounded to the nearest e2m1 value, ties to the even
 *   code, magnitudes above 6 to 6.  A block of zeros gets scale byte 0; a block that holds a NaN
 *   or an infinity gets scale byte 255 (its codes are unspecified).
 * Errors: MRR_ERR_DTYPE (dt not F16, BF16, F32), MRR_ERR_SHAPE (rows < 0, K < 2, K odd or above
 * 2^30, more than 2^31 - 1 runs of 512 elements in all, row_stride < K or above 2^31),
 * MRR_ERR_NULL, MRR_ERR_ALIGN (x not aligned to its type), MRR_ERR_CUDA.
 */
mrr_status moe_mx_quantize_run(const void *x, moe_dtype dt, int64_t rows, int64_t K, int64_t row_stride,
                               uint8_t *codes, uint8_t *scales, mrr_stream_t stream);

/*
 * moe_mx_dequantize_run -- the values of MXFP4 rows as x [rows, K] in dt (rounded to nearest where
 *   dt cannot hold one; float16 overflows to infinity).  Errors as for moe_mx_quantize_run.
 */
mrr_status moe_mx_dequantize_run(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t K,
                                 moe_dtype dt, void *x, int64_t row_stride, mrr_stream_t stream);

/* Workspace bytes of moe_mx_grouped_run for E experts (host only). */
size_t moe_mx_grouped_workspace(int64_t E);

/*
 * moe_mx_grouped_run -- the experts' product on expert-major MXFP4 rows.
 *   codes, scales   [A] rows of K elements, expert 0's rows first          (read)
 *   expert_num      [E] int32 or int64 (expert_num_is_i64): each expert's rows (expert_num_type
 *                   1), or their inclusive prefix (0), as the re-routing op writes them; zero
 *                   rows are allowed                                       (read)
 *   w_codes, w_scales  expert e's weights, [E, N, K] MXFP4, or with gated [E, 2 N, K]: N gate
 *                   rows, then N up rows                                   (read)
 *   row_weight      [A] float32, or NULL                                   (read)
 *   out             [A, N] in out_dt; row r of expert e is y[n] = sum_k x[r, k] w[e, n, k], or
 *                   with gated silu(y_gate[n]) * y_up[n], silu(g) = g / (1 + exp(-g)); then times
 *                   row_weight[r] where given; sums in float32, one rounding at the end (written)
 *   out_scales      the scales of an MXFP4 out, else NULL                  (written)
 *   workspace       >= moe_mx_grouped_workspace(E) bytes, 256-byte aligned; status words are read
 *                   with mrr_v2_read_status: MRR_ERR_COUNT_NONPOS (a negative count),
 *                   MRR_ERR_COUNT_SUM (the counts do not sum to A), MRR_ERR_TIMEOUT; the outputs
 *                   are then unspecified
 * Host errors: MRR_ERR_DTYPE, MRR_ERR_ATTR (expert_num_type, gated not 0 or 1), MRR_ERR_SHAPE (A
 * < 0 or above 2^31 - 257, E outside 1 .. 4096, K < 32 or not a multiple of 32 or above 2^20, N
 * outside 1 .. 2^20, more than 2^31 - 513 weight rows in all, an MXFP4 out with N not a multiple of
 * 32), MRR_ERR_NULL, MRR_ERR_ALIGN (codes
 * or w_codes not 16-byte aligned, scales or w_scales not 2-byte aligned, another pointer not
 * aligned to its type), MRR_ERR_WORKSPACE, MRR_ERR_CUDA.
 */
mrr_status moe_mx_grouped_run(const uint8_t *codes, const uint8_t *scales, int64_t A, int64_t K,
                              const void *expert_num, int expert_num_is_i64, int64_t expert_num_type, int64_t E,
                              const uint8_t *w_codes, const uint8_t *w_scales, int64_t N, int gated,
                              const float *row_weight, void *out, moe_dtype out_dt, uint8_t *out_scales,
                              void *workspace, size_t workspace_bytes, mrr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MX_H */
