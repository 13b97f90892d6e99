// The gradient of the root-mean-square norm (include/moe_norm.h).
//
// With g = grad_y weight, r = 1 / sqrt(mean(h^2) + eps):
//   grad_x = r g - h r^3 sum(g h) / H + grad_h,      grad_weight = sum over rows of grad_y h r
// Both sums over a row are of h and grad_y as they come from memory, so a row is read once, stays in registers,
// and one joint sum over the block gives r and the other factor.  HBM bounds it.  The blocks stay for many
// rows and hold their share of grad_weight in registers; each leaves one row of partial sums, which a second
// launch adds in order.
#include <string.h>

#include "column_sum.cuh"
#include "moe_norm.h"

using namespace moe_rows;

namespace {

constexpr int kMaxBlocks = 304;   // two on each of the 152 SMs
constexpr int kMaxWarps = 32;
constexpr int kShortWarps = 8;    // rows of a block at once where a warp has a row

struct Params {
    const void *grad_y, *h, *grad_h, *weight;
    void *grad_x;
    float *partial;        // [blocks][H], or NULL
    int64_t T;
    int H, weight_f32;
    float eps;
};

template <int DT, int W, int NV, bool kBlock>
__global__ void __launch_bounds__(kBlock ? (NV > 4 ? 1024 : NV > 2 ? 512 : 1024) : 32 * kShortWarps) rms_norm_grad(Params p)
{
    __shared__ float2 sums[2][kMaxWarps];
    extern __shared__ float shares[];   // short rows: each warp's share of grad_weight
    mrr::grid_launch_dependents();
    constexpr int kElem = DT == MOE_F32 ? 4 : 2;
    const int threads = kBlock ? blockDim.x : 32, tid = kBlock ? threadIdx.x : threadIdx.x % 32;
    const int warp = threadIdx.x / 32;
    const int64_t step = kBlock ? gridDim.x : gridDim.x * kShortWarps;
    float acc[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            acc[i][j] = 0.0f;
    int turn = 0;
    for (int64_t row = kBlock ? blockIdx.x : blockIdx.x * kShortWarps + warp; row < p.T; row += step, turn ^= 1) {
        const int64_t at = row * p.H * kElem;
        float h[NV][8], g[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (tid + i * threads);
            load8<DT, W>(static_cast<const uint8_t *>(p.h) + at, c, p.H - c, h[i]);
            load8<DT, W>(static_cast<const uint8_t *>(p.grad_y) + at, c, p.H - c, g[i]);
        }
        float squares = 0.0f, inner = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (tid + i * threads);
            float w[8];
            if (p.weight_f32)
                load8<MOE_F32, W == 2 ? 4 : W>(p.weight, c, p.H - c, w);
            else
                load8<DT, W>(p.weight, c, p.H - c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                squares = fmaf(h[i][j], h[i][j], squares);
                inner = fmaf(g[i][j] * w[j], h[i][j], inner);
            }
        }
        squares = warp_sum(squares);
        inner = warp_sum(inner);
        if (kBlock) {
            // two sets of words in turn: one barrier a row
            if (threadIdx.x % 32 == 0)
                sums[turn][warp] = make_float2(squares, inner);
            __syncthreads();
            squares = inner = 0.0f;
            for (int w = 0; w < blockDim.x / 32; ++w) {
                squares += sums[turn][w].x;
                inner += sums[turn][w].y;
            }
        }
        const float r = 1.0f / sqrtf(squares / (float)p.H + p.eps);
        const float factor = r * r * r * (inner / (float)p.H);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (tid + i * threads);
            float w[8], d[8];
            if (p.weight_f32)
                load8<MOE_F32, W == 2 ? 4 : W>(p.weight, c, p.H - c, w);
            else
                load8<DT, W>(p.weight, c, p.H - c, w);
            if (p.grad_h) {
                load8<DT, W>(static_cast<const uint8_t *>(p.grad_h) + at, c, p.H - c, d);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    d[j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                acc[i][j] = fmaf(g[i][j], h[i][j] * r, acc[i][j]);
                d[j] += r * (g[i][j] * w[j]) - h[i][j] * factor;
            }
            store8<DT, W>(static_cast<uint8_t *>(p.grad_x) + at, c, p.H - c, d);
        }
    }
    if (!p.partial)
        return;
    float *to = p.partial + (int64_t)blockIdx.x * p.H;
    if (kBlock) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (8 * (tid + i * threads) + j < p.H)
                    to[8 * (tid + i * threads) + j] = acc[i][j];
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (8 * (tid + i * threads) + j < p.H)
                    shares[warp * p.H + 8 * (tid + i * threads) + j] = acc[i][j];
        __syncthreads();
        for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kShortWarps; ++w)
                s += shares[w * p.H + c];
            to[c] = s;
        }
    }
}

int64_t blocks_for(int64_t T, int64_t H)
{
    const int64_t rows = H <= 1024 ? kShortWarps : 1, blocks = (T + rows - 1) / rows;
    return blocks < kMaxBlocks ? blocks : kMaxBlocks;
}

template <int DT, int W>
void launch(const Params &p, cudaStream_t st)
{
    const int chunks = (p.H + 7) / 8;
    const unsigned grid = (unsigned)blocks_for(p.T, p.H);
    auto threads = [&](int each) { return (unsigned)(((chunks + each - 1) / each + 31) / 32 * 32); };
    if (chunks <= 32)
        rms_norm_grad<DT, W, 1, false><<<grid, 32 * kShortWarps, kShortWarps * p.H * 4, st>>>(p);
    else if (chunks <= 128)
        rms_norm_grad<DT, W, 4, false><<<grid, 32 * kShortWarps, kShortWarps * p.H * 4, st>>>(p);
    else if (chunks <= 2048)
        rms_norm_grad<DT, W, 4, true><<<grid, threads(4), 0, st>>>(p);
    else
        rms_norm_grad<DT, W, 8, true><<<grid, threads(8), 0, st>>>(p);
}

template <int DT>
void launch(const Params &p, uintptr_t all, cudaStream_t st)
{
    if (all % 16 == 0)
        launch<DT, 16>(p, st);
    else if (all % 8 == 0)
        launch<DT, 8>(p, st);
    else if (all % 4 == 0 || DT == MOE_F32)
        launch<DT, 4>(p, st);
    else
        launch<DT, DT == MOE_F32 ? 4 : 2>(p, st);
}

bool aligned(const void *p, uintptr_t n) { return (uintptr_t)p % n == 0; }
uintptr_t size_of(int dt) { return dt == MOE_F32 ? 4 : 2; }
bool is_float(int dt) { return dt == MOE_F16 || dt == MOE_BF16 || dt == MOE_F32; }

}  // namespace

extern "C" {

size_t moe_add_rms_norm_grad_workspace(int64_t T, int64_t H)
{
    if (T < 0 || T > INT32_MAX || H < 1 || H > MOE_NORM_MAX_H)
        return 0;
    return (size_t)((blocks_for(T, H) * H * 4 + 255) / 256 * 256);
}

mrr_status moe_add_rms_norm_grad_run(const void *grad_y, const void *h, const void *grad_h, moe_dtype dt, int64_t T,
                                     int64_t H, const void *weight, moe_dtype weight_dt, float eps, void *grad_x,
                                     void *grad_weight, void *workspace, size_t workspace_bytes, mrr_stream_t stream)
{
    if (!is_float(dt) || (weight_dt != dt && weight_dt != MOE_F32))
        return MRR_ERR_DTYPE;
    if (!(eps >= 0.0f))
        return MRR_ERR_ATTR;
    if (T < 0 || T > INT32_MAX || H < 1 || H > MOE_NORM_MAX_H)
        return MRR_ERR_SHAPE;
    if (!weight || (T > 0 && (!grad_y || !h || !grad_x)))
        return MRR_ERR_NULL;
    const uintptr_t size = size_of(dt);
    if (!aligned(grad_y, size) || !aligned(h, size) || !aligned(grad_h, size) || !aligned(grad_x, size) ||
        !aligned(weight, size_of(weight_dt)) || !aligned(grad_weight, size_of(weight_dt)))
        return MRR_ERR_ALIGN;
    if (grad_weight && T > 0 &&
        (!workspace || !aligned(workspace, 256) || workspace_bytes < moe_add_rms_norm_grad_workspace(T, H)))
        return MRR_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (T > 0) {
        Params p;
        memset(&p, 0, sizeof(p));
        p.grad_y = grad_y;
        p.h = h;
        p.grad_h = grad_h;
        p.weight = weight;
        p.grad_x = grad_x;
        p.partial = grad_weight ? static_cast<float *>(workspace) : nullptr;
        p.T = T;
        p.H = (int)H;
        p.weight_f32 = weight_dt == MOE_F32;
        p.eps = eps;
        const uintptr_t all = (uintptr_t)grad_y | (uintptr_t)h | (uintptr_t)grad_h | (uintptr_t)grad_x |
                              (uintptr_t)weight | (T > 1 ? (uintptr_t)H * size : 0);
        if (dt == MOE_F32)
            launch<MOE_F32>(p, all, st);
        else if (dt == MOE_BF16)
            launch<MOE_BF16>(p, all, st);
        else
            launch<MOE_F16>(p, all, st);
        if (cudaGetLastError() != cudaSuccess)
            return MRR_ERR_CUDA;
    }
    if (grad_weight && launch_column_sum(static_cast<const float *>(workspace), T > 0 ? (int)blocks_for(T, H) : 0, H,
                                         (int)H, weight_dt, grad_weight, st) != cudaSuccess) {
        (void)cudaGetLastError();
        return MRR_ERR_CUDA;
    }
    return MRR_OK;
}

}  // extern "C"
