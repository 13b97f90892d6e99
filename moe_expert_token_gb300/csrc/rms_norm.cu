// Host entry points of the norm and its gradient, and rows of 8 bits back to values (include/moe_norm.h).  The norm's
// kernels are in rms_norm_kernel.cuh and rms_norm_grad_kernel.cuh.
#include <string.h>

#include "column_sum.cuh"
#include "rms_norm.h"
#include "rows.cuh"

using namespace moe_rows;
using namespace moe_norm;

namespace {

// Rows of 8 bits back to values.  Rows that are multiples of 8 elements, on aligned addresses, are taken by groups of
// threads, each with kAtOnce chunks of 8 elements under way.
constexpr int kThreads = 128, kAtOnce = 4;

struct Values {
    const uint8_t *q;
    const void *scales;
    void *x;
    int64_t T;
    int H, quant, chunks, group, rows;   // threads of a row, rows of a block
};

__device__ __forceinline__ float scale_of(const Values &p, int64_t row, int at)
{
    if (p.quant == MOE_Q_MXFP8)
        return e8m0_value(__ldg(static_cast<const uint8_t *>(p.scales) + row * ((p.H + 63) / 64 * 2) + at / 32));
    if (p.quant == MOE_Q_E4M3_128)
        return __ldg(static_cast<const float *>(p.scales) + row * ((p.H + 127) / 128) + at / 128);
    return __ldg(static_cast<const float *>(p.scales) + row);
}

__device__ __forceinline__ float2 values_of(const Values &p, uint2 codes, int i)
{
    const uint32_t two = (i < 4 ? codes.x : codes.y) >> (8 * (i % 4)) & 0xffffu;
    return p.quant == MOE_Q_INT8 ? make_float2((float)(int8_t)two, (float)(int8_t)(two >> 8)) : decode_e4m3x2(two);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) dequantize(Values p)
{
    const int of_block = threadIdx.x / p.group, lane = threadIdx.x - of_block * p.group;
    const int64_t row = (int64_t)blockIdx.x * p.rows + of_block;
    if (row >= p.T)
        return;
    const uint2 *from = reinterpret_cast<const uint2 *>(p.q + row * p.H);
    using C = Chunk<DT, 16>;
    uint8_t *to = static_cast<uint8_t *>(p.x) + row * p.H * C::kElem;
    const bool by_row = p.quant == MOE_Q_INT8 || p.quant == MOE_Q_E4M3;
    const float of_row = by_row ? scale_of(p, row, 0) : 0.0f;
    for (int c0 = lane; c0 < p.chunks; c0 += kAtOnce * p.group) {
        uint2 w[kAtOnce];
        float s[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int c = c0 + u * p.group;
            w[u] = c < p.chunks ? __ldg(from + c) : make_uint2(0u, 0u);
            s[u] = of_row;
        }
        if (!by_row) {   // (apart: a branch between the loads keeps them from being under way together)
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)
                s[u] = c0 + u * p.group < p.chunks ? scale_of(p, row, 8 * (c0 + u * p.group)) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int c = c0 + u * p.group;
            if (c >= p.chunks)
                continue;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 f = values_of(p, w[u], i);
                v[i] = f.x * s[u], v[i + 1] = f.y * s[u];
            }
            C out;
            out.set(v);
            out.store(to, c * C::kBytes, p.H * C::kElem);
        }
    }
}

// Rows of any size: all codes are one array without gaps and so are the values, so a thread takes 8 of them that begin
// at a multiple of 8 wherever the rows begin (kWide: on aligned addresses).  Where they all have one scale it is
// looked up once.
template <int DT, bool kWide>
__global__ void __launch_bounds__(kThreads) dequantize_flat(Values p)
{
    const int64_t all = p.T * p.H, first = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8;
    if (first >= all)
        return;
    const int n = (int)min((int64_t)8, all - first);
    uint2 w = make_uint2(0u, 0u);
    if (kWide && n == 8) {
        w = __ldg(reinterpret_cast<const uint2 *>(p.q + first));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                (i < 4 ? w.x : w.y) |= (uint32_t)__ldg(p.q + first + i) << (8 * (i % 4));
    }
    const int64_t row = first / p.H;
    const int at = (int)(first - row * p.H);
    const int block = p.quant == MOE_Q_MXFP8 ? 32 : p.quant == MOE_Q_E4M3_128 ? 128 : p.H;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 f = values_of(p, w, i);
        v[i] = f.x, v[i + 1] = f.y;
    }
    float s = scale_of(p, row, at);
    if (at / block == (at + 7) / block && at + 8 <= p.H) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] *= s;
    } else {
        int64_t r = row;
        int c = at, left = min(p.H - at, block - at % block);   // elements with this scale
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= n)
                break;
            if (left == 0) {
                c = c == p.H ? 0 : c;
                r += c == 0;
                left = min(p.H - c, block);
                s = scale_of(p, r, c);
            }
            v[i] *= s;
            ++c;
            --left;
        }
    }
    constexpr int kElem = DT == MOE_F32 ? 4 : 2;
    Chunk<DT, kWide ? 16 : kElem> out;
    out.set(v);
    if (kWide && n < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                store1<DT>(p.x, first + i, v[i]);
    } else {
        out.store(static_cast<uint8_t *>(p.x) + first * kElem, 0, n * kElem);
    }
}

bool aligned(const void *p, uintptr_t n) { return (uintptr_t)p % n == 0; }
uintptr_t size_of(int dt) { return dt == MOE_F32 ? 4 : 2; }
bool is_float(int dt) { return dt == MOE_F16 || dt == MOE_BF16 || dt == MOE_F32; }

mrr_status done(cudaError_t err)
{
    if (err == cudaSuccess)
        return MRR_OK;
    (void)cudaGetLastError();
    return MRR_ERR_CUDA;
}

}  // namespace

extern "C" {

mrr_status moe_add_rms_norm_run(const void *x, const void *residual, moe_dtype dt, int64_t T, int64_t H,
                                int64_t x_stride, int64_t residual_stride, const void *weight, moe_dtype weight_dt,
                                float eps, void *h, void *y, moe_quant quant, void *q, void *scales,
                                mrr_stream_t stream)
{
    if (!is_float(dt) || (weight_dt != dt && weight_dt != MOE_F32))
        return MRR_ERR_DTYPE;
    if (quant < MOE_Q_NONE || quant > MOE_Q_MXFP4 || !(eps >= 0.0f))
        return MRR_ERR_ATTR;
    if (T < 0 || T > INT32_MAX || H < 1 || H > MOE_NORM_MAX_H || x_stride < H || x_stride > (1ll << 31) ||
        (residual && (residual_stride < H || residual_stride > (1ll << 31))) || (quant == MOE_Q_MXFP4 && H % 2))
        return MRR_ERR_SHAPE;
    if (!weight || (T > 0 && (!x || (!h && !y && quant == MOE_Q_NONE) || (quant != MOE_Q_NONE && (!q || !scales)))))
        return MRR_ERR_NULL;
    const uintptr_t size = size_of(dt);
    if (!aligned(x, size) || (residual && !aligned(residual, size)) || !aligned(weight, size_of(weight_dt)) ||
        (h && !aligned(h, size)) || (y && !aligned(y, size)) ||
        (quant != MOE_Q_NONE && quant < MOE_Q_MXFP8 && !aligned(scales, 4)))
        return MRR_ERR_ALIGN;
    if (T == 0)
        return MRR_OK;
    Params p;
    memset(&p, 0, sizeof(p));
    p.x = x;
    p.residual = residual;
    p.weight = weight;
    p.h = h;
    p.y = y;
    p.q = q;
    p.scales = scales;
    p.T = T;
    p.x_stride = x_stride;
    p.residual_stride = residual_stride;
    p.H = (int)H;
    p.weight_f32 = weight_dt == MOE_F32;
    p.quant = quant;
    const uintptr_t codes = (uintptr_t)q | (uintptr_t)(quant == MOE_Q_MXFP4 ? H / 2 : H);
    p.q_align = codes % 8 == 0 ? 8 : codes % 4 == 0 ? 4 : codes % 2 == 0 ? 2 : 1;
    p.eps = eps;
    // pieces that every row begins with and consists of
    uintptr_t all = (uintptr_t)x | (uintptr_t)weight | (uintptr_t)h | (uintptr_t)y | (uintptr_t)H * size;
    if (T > 1)
        all |= (uintptr_t)x_stride * size | (residual ? (uintptr_t)residual_stride * size : 0);
    if (residual)
        all |= (uintptr_t)residual;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return done(dt == MOE_F32 ? norm_f32(p, all, st) : dt == MOE_BF16 ? norm_bf16(p, all, st) : norm_f16(p, all, st));
}

mrr_status moe_dequantize_rows_run(const void *q, const void *scales, moe_quant quant, int64_t T, int64_t H,
                                   moe_dtype dt, void *x, mrr_stream_t stream)
{
    if (!is_float(dt))
        return MRR_ERR_DTYPE;
    if (quant < MOE_Q_INT8 || quant > MOE_Q_MXFP8)
        return MRR_ERR_ATTR;
    if (T < 0 || T > INT32_MAX || H < 1 || H > (1 << 20))
        return MRR_ERR_SHAPE;
    if (T > 0 && (!q || !scales || !x))
        return MRR_ERR_NULL;
    if (!aligned(x, size_of(dt)) || (quant != MOE_Q_MXFP8 && !aligned(scales, 4)))
        return MRR_ERR_ALIGN;
    if (T == 0)
        return MRR_OK;
    Values p;
    memset(&p, 0, sizeof(p));
    p.q = static_cast<const uint8_t *>(q);
    p.scales = scales;
    p.x = x;
    p.T = T;
    p.H = (int)H;
    p.quant = quant;
    const bool wide = aligned(q, 8) && aligned(x, 16);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!wide || H % 8) {
        const int64_t blocks = (T * H + 8 * kThreads - 1) / (8 * kThreads);
        if (blocks > INT32_MAX)
            return MRR_ERR_SHAPE;
        auto kernel = dt == MOE_F32    ? (wide ? dequantize_flat<MOE_F32, true> : dequantize_flat<MOE_F32, false>)
                      : dt == MOE_BF16 ? (wide ? dequantize_flat<MOE_BF16, true> : dequantize_flat<MOE_BF16, false>)
                                       : (wide ? dequantize_flat<MOE_F16, true> : dequantize_flat<MOE_F16, false>);
        kernel<<<(unsigned)blocks, kThreads, 0, st>>>(p);
        return done(cudaGetLastError());
    }
    p.chunks = (int)(H / 8);
    // many rows: as many threads as have kAtOnce chunks each; few: as have one.  A power of two up to 16, else warps.
    const int64_t each = T < 2 * 152 ? 1 : kAtOnce, need = (p.chunks + each - 1) / each;
    p.group = need > 16 ? (int)(need < kThreads ? (need + 31) / 32 * 32 : kThreads) : 1;
    while (need <= 16 && p.group < need)
        p.group *= 2;
    p.rows = kThreads / p.group;
    const unsigned grid = (unsigned)((T + p.rows - 1) / p.rows), threads = p.group * p.rows;
    auto kernel = dt == MOE_F32 ? dequantize<MOE_F32> : dt == MOE_BF16 ? dequantize<MOE_BF16> : dequantize<MOE_F16>;
    kernel<<<grid, threads, 0, st>>>(p);
    return done(cudaGetLastError());
}

size_t moe_add_rms_norm_grad_workspace(int64_t T, int64_t H)
{
    if (T < 0 || T > INT32_MAX || H < 1 || H > MOE_NORM_MAX_H)
        return 0;
    return (size_t)((grad_blocks(T, H) * H * 4 + 255) / 256 * 256);
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
        GradParams p;
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
                              (uintptr_t)weight | (uintptr_t)H * size;
        mrr_device::Info info;
        cudaError_t err = cudaErrorUnknown;
        if (mrr_device::current(info))
            err = dt == MOE_F32    ? norm_grad_f32(p, all, info, st)
                  : dt == MOE_BF16 ? norm_grad_bf16(p, all, info, st)
                                   : norm_grad_f16(p, all, info, st);
        if (err != cudaSuccess) {
            (void)cudaGetLastError();
            return MRR_ERR_CUDA;
        }
    }
    if (grad_weight && launch_column_sum(static_cast<const float *>(workspace), T > 0 ? (int)grad_blocks(T, H) : 0, H,
                                         (int)H, weight_dt, grad_weight, st) != cudaSuccess) {
        (void)cudaGetLastError();
        return MRR_ERR_CUDA;
    }
    return MRR_OK;
}

}  // extern "C"
