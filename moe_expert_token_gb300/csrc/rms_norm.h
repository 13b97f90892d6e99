// The norm's kernels as its host entry points see them: one translation unit for each element type.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "device_info.h"
#include "moe_norm.h"

namespace moe_norm {

struct Params {
    const void *x, *residual, *weight;
    void *h, *y, *q, *scales;
    int64_t T, x_stride, residual_stride;   // in elements
    int H, weight_f32, quant, q_align;      // q_align: of every chunk's codes, up to their size
    float eps;
};

struct GradParams {
    const void *grad_y, *h, *grad_h, *weight;
    void *grad_x;
    float *partial;        // [blocks][H], or NULL
    int64_t T;
    int H, weight_f32;
    int tensors;           // 3: grad_h comes ahead as grad_y and h do
    float eps;
};

constexpr int kShortWarps = 8;    // rows at once of the gradient's blocks where a warp has a row

// The gradient's blocks: one on each of the 152 SMs, and two where rows are many and short enough for two blocks'
// registers (300 rows of 7168: 14.4 us with 152, 16.5 with 304; 16384 rows: 158 and 148; 4000 rows of 12288: 76 and 85)
inline int64_t grad_blocks(int64_t T, int64_t H)
{
    const int64_t rows = H <= 1024 ? kShortWarps : 1, blocks = (T + rows - 1) / rows;
    const int64_t most = H > 7168 || blocks < 8 * 304 ? 152 : 304;
    return blocks < most ? blocks : most;
}

// `all`: the pieces that rows come in, in its lowest bits (every address, stride and size or-ed together)
cudaError_t norm_f16(const Params &p, uintptr_t all, cudaStream_t st);
cudaError_t norm_bf16(const Params &p, uintptr_t all, cudaStream_t st);
cudaError_t norm_f32(const Params &p, uintptr_t all, cudaStream_t st);
cudaError_t norm_grad_f16(const GradParams &p, uintptr_t all, const mrr_device::Info &info, cudaStream_t st);
cudaError_t norm_grad_bf16(const GradParams &p, uintptr_t all, const mrr_device::Info &info, cudaStream_t st);
cudaError_t norm_grad_f32(const GradParams &p, uintptr_t all, const mrr_device::Info &info, cudaStream_t st);

}  // namespace moe_norm
