// Sums over many rows of a float32 table's columns, in a fixed order: the second half of a gradient that is summed
// over tokens.  Each block of the first half leaves one row of partial sums.
#pragma once

#include "ptx.cuh"
#include "rows.cuh"

namespace moe_rows {

constexpr int kSumColumns = 32, kSumWarps = 32;

// out[c] in dt = sum over rows r < rows of table[r * pitch + c], c < columns; a warp adds every 32nd row.  Launched
// as the programmatic successor of the kernel that writes the table.
static __global__ void __launch_bounds__(kSumColumns * kSumWarps) column_sum(const float *table, int rows, int64_t pitch,
                                                                             int columns, int dt, void *out)
{
    __shared__ float part[kSumWarps][kSumColumns];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int c = blockIdx.x * kSumColumns + lane;
    mrr::grid_dependency_wait();
    float sum = 0.0f;
    if (c < columns) {
#pragma unroll 8
        for (int r = warp; r < rows; r += kSumWarps)
            sum += table[r * pitch + c];
    }
    part[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < columns) {
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kSumWarps; ++w)
            sum += part[w][lane];
        if (dt == MOE_F32)
            store1<MOE_F32>(out, c, sum);
        else if (dt == MOE_BF16)
            store1<MOE_BF16>(out, c, sum);
        else
            store1<MOE_F16>(out, c, sum);
    }
}

static inline cudaError_t launch_column_sum(const float *table, int rows, int64_t pitch, int columns, int dt, void *out,
                                            cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((columns + kSumColumns - 1) / kSumColumns);
    cfg.blockDim = dim3(kSumColumns * kSumWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, column_sum, table, rows, pitch, columns, dt, out);
}

}  // namespace moe_rows
