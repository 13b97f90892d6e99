/*
 * moe_norm.h -- C ABI of the norm in front of a mixture-of-experts block, for GB300 (sm_103a): a
 * residual's addition, the root-mean-square norm of the sum, the result also in 8 bits or MXFP4 with
 * the scales that the re-routing op moves, rows of 8 bits back to values, and the norm's gradient.
 *
 *   h[t, c] = x[t, c] + residual[t, c]                              (float32)
 *   r[t]    = 1 / sqrt(sum_c h[t, c]^2 / H + eps)
 *   y[t, c] = h[t, c] r[t] weight[c]                                (float32 up to its one rounding)
 * y is made from h before h is rounded to be stored, the quantised rows from y before it is.  The sum is float32 too: of a row
 * whose squares add up to more than that holds (elements of 2^64 / sqrt(H) or more) r is 0, of one whose squares are 0 in it under an
 * eps of 0 r is infinite, in the gradient as well.
 *
 * Quantised rows, q with scales; m is the largest magnitude of y's row or block:
 *   MOE_Q_INT8      int8;  scales [T] float32           s = m / 127, q = y / s to nearest even
 *   MOE_Q_E4M3      e4m3;  scales [T] float32           s = m / 448
 *   MOE_Q_E4M3_128  e4m3;  scales [T, ceil(H/128)] float32, one for each 128 elements, s = m / 448
 *   MOE_Q_MXFP8     e4m3;  scales [T, ceil(H/64), 2] e8m0, one for each 32 elements:
 *                   2^(floor(log2 m) - 8), the exponent held to -127 .. 127
 *   MOE_Q_MXFP4     e2m1 codes [T, H/2] and e8m0 scales [T, ceil(H/64), 2], as moe_mx_quantize_run
 *                   makes them of y in float32
 * Float32 scales are held to 2^-126 from below.  An element is y / s rounded to nearest, ties to
 * even, magnitudes above the type's largest to that; y / s itself is rounded to float32.  A row or
 * block that holds a NaN or an infinity gets the scale NaN (e8m0: 255), its codes are unspecified;
 * where the last e8m0 pair has no second block its byte is written as 127 and never used.
 *
 * Conventions are those of mrr_v2.h.  The same inputs give the same bits; a row's last bits may differ with the number
 * of rows beside it, as how its sum is shared out does.  Calls that may run at the same time need workspaces of their
 * own.  Calls may be captured in a CUDA graph.
 */
#ifndef MOE_NORM_H
#define MOE_NORM_H

#include "moe_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_quant {
    MOE_Q_NONE = 0,
    MOE_Q_INT8 = 1,
    MOE_Q_E4M3 = 2,
    MOE_Q_E4M3_128 = 3,
    MOE_Q_MXFP8 = 4,
    MOE_Q_MXFP4 = 5
} moe_quant;

/* largest row of the norm */
#define MOE_NORM_MAX_H 65536

/*
 * moe_add_rms_norm_run
 *   x        [T, H] in dt (F16, BF16, F32), row t at x + t * x_stride elements            (read)
 *   residual [T, H] in dt, row stride residual_stride, or NULL                            (read)
 *   weight   [H] in weight_dt: dt or F32                                                  (read)
 *   h        [T, H] in dt without gaps; NULL without residual, or where it is not wanted  (written)
 *   y        [T, H] in dt without gaps; NULL where only quantised rows are wanted         (written)
 *   q, scales  as above; NULL for MOE_Q_NONE                                              (written)
 * Host errors: MRR_ERR_DTYPE, MRR_ERR_ATTR (quant, eps negative or NaN), MRR_ERR_SHAPE (T < 0 or
 * above 2^31 - 1, H outside 1 .. 65536, odd H with MXFP4, a stride < H or above 2^31), MRR_ERR_NULL (no
 * output at all, ...), MRR_ERR_ALIGN (a pointer not aligned to its type), MRR_ERR_CUDA.
 */
mrr_status moe_add_rms_norm_run(const void *x, const void *residual, moe_dtype dt, int64_t T, int64_t H,
                                int64_t x_stride, int64_t residual_stride, const void *weight, moe_dtype weight_dt,
                                float eps, void *h, void *y, moe_quant quant, void *q, void *scales,
                                mrr_stream_t stream);

/* Workspace bytes of moe_add_rms_norm_grad_run (host only); 0 where a size is out of range. */
size_t moe_add_rms_norm_grad_workspace(int64_t T, int64_t H);

/*
 * moe_add_rms_norm_grad_run -- the gradient of y (and h) with respect to x (and, as it is the same,
 *   residual) and weight:
 *   g = grad_y weight, u = h r, grad_x = r (g - u sum_c(g u) / H) + grad_h
 *   grad_weight[c] = sum over t of grad_y[t, c] u[t, c]
 *   in float32, each rounded once.  h is what moe_add_rms_norm_run stored (x without a residual).
 *   grad_y, h, grad_h (or NULL) [T, H] in dt without gaps; weight [H] in weight_dt         (read)
 *   grad_x [T, H] in dt; grad_weight [H] in weight_dt, or NULL                             (written)
 *   workspace  >= moe_add_rms_norm_grad_workspace(T, H) bytes, 256-byte aligned; not initialised
 * Host errors as for moe_add_rms_norm_run, and MRR_ERR_WORKSPACE.
 */
mrr_status moe_add_rms_norm_grad_run(const void *grad_y, const void *h, const void *grad_h, moe_dtype dt, int64_t T,
                                     int64_t H, const void *weight, moe_dtype weight_dt, float eps, void *grad_x,
                                     void *grad_weight, void *workspace, size_t workspace_bytes, mrr_stream_t stream);

/*
 * moe_dequantize_rows_run -- the values [T, H] in dt of quantised rows (MOE_Q_INT8, MOE_Q_E4M3,
 *   MOE_Q_E4M3_128 or MOE_Q_MXFP8; MXFP4 rows: moe_mx_dequantize_run), code times scale in
 *   float32, rounded once.
 * Host errors: MRR_ERR_DTYPE, MRR_ERR_ATTR (quant), MRR_ERR_SHAPE (T < 0 or above 2^31 - 1, more than 2^41 elements, H
 * outside 1 .. 2^20), MRR_ERR_NULL, MRR_ERR_ALIGN, MRR_ERR_CUDA.
 */
mrr_status moe_dequantize_rows_run(const void *q, const void *scales, moe_quant quant, int64_t T, int64_t H,
                                   moe_dtype dt, void *x, mrr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_NORM_H */
