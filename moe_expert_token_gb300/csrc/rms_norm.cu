// A residual's addition, the root-mean-square norm of the sum with its 8-bit and MXFP4 forms, and rows of 8 bits
// back to values (include/moe_norm.h).
//
// h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight: every element is read and written once and a
// handful of operations are made of it, so HBM bounds both.  A row stays in registers, 8 elements a
// chunk, between the sum of its squares and the results: it belongs to one block (or, where it is short,
// to one warp).
#include <string.h>

#include "moe_norm.h"
#include "rows.cuh"

using namespace moe_rows;

namespace {

constexpr int kMaxWarps = 32;

struct Params {
    const void *x, *residual, *weight;
    void *h, *y, *q, *scales;
    int64_t T, x_stride, residual_stride;   // in elements
    int H, weight_f32, quant, q_wide;       // q_wide: a chunk's codes are stored at once
    float eps;
};

// The sum or maximum of v over the row's threads: a warp's, or with kBlock all warps'; each thread gets it.
template <bool kBlock>
__device__ __forceinline__ float row_sum(float v, float *of_warp)
{
    v = warp_sum(v);
    if (kBlock) {
        if (threadIdx.x % 32 == 0)
            of_warp[threadIdx.x / 32] = v;
        __syncthreads();
        v = 0.0f;
        for (int w = 0; w < blockDim.x / 32; ++w)
            v += of_warp[w];
    }
    return v;
}

template <bool kBlock>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *of_warp)
{
    v = __reduce_max_sync(kFull, v);
    if (kBlock) {
        if (threadIdx.x % 32 == 0)
            of_warp[threadIdx.x / 32] = v;
        __syncthreads();
        v = 0u;
        for (int w = 0; w < blockDim.x / 32; ++w)
            v = max(v, of_warp[w]);
    }
    return v;
}

// the float32 scale of magnitudes up to the float with bits m, for codes up to `top`, and its reciprocal
__device__ __forceinline__ float float_scale(uint32_t m, float top, float &inverse)
{
    if (m >= 0x7f800000u) {
        inverse = 0.0f;
        return __uint_as_float(0x7fffffffu);
    }
    const float s = fmaxf(__uint_as_float(m) / top, 0x1p-126f);
    inverse = 1.0f / s;
    return s;
}

__device__ __forceinline__ uint32_t int8_of(float v) { return (uint32_t)min(127, max(-127, __float2int_rn(v))) & 0xffu; }

// codes of a chunk (elements c .. c + n - 1 of row `row`), from their values over the scale
__device__ __forceinline__ void store_bytes(const Params &p, int64_t row, int c, int n, uint32_t lo, uint32_t hi)
{
    uint8_t *to = static_cast<uint8_t *>(p.q) + row * p.H + c;
    if (n >= 8 && p.q_wide) {
        *reinterpret_cast<uint2 *>(to) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                to[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i % 4)));
    }
}

__device__ __forceinline__ uint32_t largest(const float (&v)[8])
{
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

// y's chunks of one row to codes and scales.  A block of 32 elements is 4 lanes' chunks, one of 128 elements 16 lanes'.
template <int NV, bool kBlock>
__device__ __forceinline__ void quantize(const Params &p, int64_t row, int tid, int threads, const float (&y)[NV][8],
                                         uint32_t *of_warp)
{
    const int kind = p.quant;
    if (kind == MOE_Q_INT8 || kind == MOE_Q_E4M3) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            m = max(m, largest(y[i]));
        m = row_max<kBlock>(m, of_warp);
        float inverse;
        const float s = float_scale(m, kind == MOE_Q_INT8 ? 127.0f : 448.0f, inverse);
        if (tid == 0)
            static_cast<float *>(p.scales)[row] = s;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (tid + i * threads), n = p.H - c;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = y[i][j] * inverse;
            if (n <= 0)
                continue;
            if (kind == MOE_Q_INT8)
                store_bytes(p, row, c, n, int8_of(v[0]) | int8_of(v[1]) << 8 | int8_of(v[2]) << 16 | int8_of(v[3]) << 24,
                            int8_of(v[4]) | int8_of(v[5]) << 8 | int8_of(v[6]) << 16 | int8_of(v[7]) << 24);
            else
                store_bytes(p, row, c, n, encode_e4m3(v[0], v[1], v[2], v[3]), encode_e4m3(v[4], v[5], v[6], v[7]));
        }
        return;
    }
    const int blocks = (p.H + 31) / 32;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = 8 * (tid + i * threads), n = p.H - c;
        uint32_t m = largest(y[i]);
        m = max(m, __shfl_xor_sync(kFull, m, 1));
        m = max(m, __shfl_xor_sync(kFull, m, 2));
        float inverse;
        if (kind == MOE_Q_E4M3_128) {
            m = max(m, __shfl_xor_sync(kFull, m, 4));
            m = max(m, __shfl_xor_sync(kFull, m, 8));
            const float s = float_scale(m, 448.0f, inverse);
            if (c % 128 == 0 && n > 0)
                static_cast<float *>(p.scales)[row * ((p.H + 127) / 128) + c / 128] = s;
        } else {
            // the exponent field of m is floor(log2 m) + 127; 8 (e4m3) or 2 (e2m1) less is the scale's byte
            const uint32_t less = kind == MOE_Q_MXFP8 ? 8u : 2u, field = m >> 23;
            const uint32_t b = field == 255u ? 255u : field > less ? field - less : 0u;
            inverse = __uint_as_float((254u - min(b, 252u)) << 23);
            if (c % 32 == 0 && n > 0) {
                uint8_t *to = static_cast<uint8_t *>(p.scales) + row * ((p.H + 63) / 64 * 2) + c / 32;
                to[0] = (uint8_t)b;
                if (c / 32 == blocks - 1 && blocks % 2)
                    to[1] = 127u;
            }
        }
        if (n <= 0)
            continue;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = y[i][j] * inverse;
        if (kind == MOE_Q_MXFP4) {
            const uint32_t w = encode8(v);
            uint8_t *to = static_cast<uint8_t *>(p.q) + (row * p.H + c) / 2;
            if (n >= 8 && p.q_wide) {
                *reinterpret_cast<uint32_t *>(to) = w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (2 * j < n)
                        to[j] = (uint8_t)(w >> (8 * j));
            }
        } else {
            store_bytes(p, row, c, n, encode_e4m3(v[0], v[1], v[2], v[3]), encode_e4m3(v[4], v[5], v[6], v[7]));
        }
    }
}

// NV chunks a thread; kBlock: a block has a row, else each of its warps has one.
template <int DT, int W, int NV, bool kBlock>
__global__ void __launch_bounds__(kBlock ? 1024 : 256) add_rms_norm(Params p)
{
    __shared__ float sums[kMaxWarps];
    __shared__ uint32_t tops[kMaxWarps];
    const int threads = kBlock ? blockDim.x : 32, tid = kBlock ? threadIdx.x : threadIdx.x % 32;
    const int64_t row = kBlock ? blockIdx.x : (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    if (row >= p.T)
        return;
    constexpr int kElem = DT == MOE_F32 ? 4 : 2;
    const uint8_t *x = static_cast<const uint8_t *>(p.x) + row * p.x_stride * kElem;
    const uint8_t *res = static_cast<const uint8_t *>(p.residual) + row * p.residual_stride * kElem;
    float v[NV][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = 8 * (tid + i * threads);
        load8<DT, W>(x, c, p.H - c, v[i]);
    }
    if (p.residual) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (tid + i * threads);
            float r[8];
            load8<DT, W>(res, c, p.H - c, r);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] += r[j];
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = 8 * (tid + i * threads);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum = fmaf(v[i][j], v[i][j], sum);
        if (p.h)
            store8<DT, W>(static_cast<uint8_t *>(p.h) + row * p.H * kElem, c, p.H - c, v[i]);
    }
    sum = row_sum<kBlock>(sum, sums);
    const float r = 1.0f / sqrtf(sum / (float)p.H + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = 8 * (tid + i * threads);
        float w[8];
        if (p.weight_f32)
            load8<MOE_F32, W == 2 ? 4 : W>(p.weight, c, p.H - c, w);
        else
            load8<DT, W>(p.weight, c, p.H - c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[i][j] = v[i][j] * r * w[j];
        if (p.y)
            store8<DT, W>(static_cast<uint8_t *>(p.y) + row * p.H * kElem, c, p.H - c, v[i]);
    }
    if (p.quant != MOE_Q_NONE)
        quantize<NV, kBlock>(p, row, tid, threads, v, tops);
}

template <int DT, int W>
void launch(const Params &p, cudaStream_t st)
{
    const int chunks = (p.H + 7) / 8;
    // Short rows: a warp each.
    if (chunks <= 128) {
        const unsigned grid = (unsigned)((p.T + 7) / 8);
        if (chunks <= 32)
            add_rms_norm<DT, W, 1, false><<<grid, 256, 0, st>>>(p);
        else
            add_rms_norm<DT, W, 4, false><<<grid, 256, 0, st>>>(p);
        return;
    }
    // Few rows: as many threads to a row as there are chunks.  Many: four chunks a thread.
    auto threads = [&](int each) { return (unsigned)(((chunks + each - 1) / each + 31) / 32 * 32); };
    const unsigned grid = (unsigned)p.T;
    if (p.T <= 304 && chunks <= 1024)
        add_rms_norm<DT, W, 1, true><<<grid, threads(1), 0, st>>>(p);
    else if (chunks <= 4096)
        add_rms_norm<DT, W, 4, true><<<grid, threads(4), 0, st>>>(p);
    else
        add_rms_norm<DT, W, 8, true><<<grid, threads(8), 0, st>>>(p);
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

// Rows of 8 bits back to values: a thread has 8 elements of one row.
template <int DT>
__global__ void __launch_bounds__(256) dequantize(const uint8_t *q, const void *scales, int kind, int64_t T, int H,
                                                  int chunks, int wide, void *x)
{
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = at / chunks;
    if (row >= T)
        return;
    const int c = (int)(at - row * chunks) * 8, n = min(8, H - c);
    const uint8_t *from = q + row * H + c;
    uint32_t w[2] = {0u, 0u};
    if (wide) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(from));
        w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                w[i / 4] |= (uint32_t)__ldg(from + i) << (8 * (i % 4));
    }
    float s;
    if (kind == MOE_Q_MXFP8)
        s = e8m0_value(__ldg(static_cast<const uint8_t *>(scales) + row * ((H + 63) / 64 * 2) + c / 32));
    else if (kind == MOE_Q_E4M3_128)
        s = __ldg(static_cast<const float *>(scales) + row * ((H + 127) / 128) + c / 128);
    else
        s = __ldg(static_cast<const float *>(scales) + row);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint32_t two = w[i / 4] >> (8 * (i % 4)) & 0xffffu;
        const float2 f = kind == MOE_Q_INT8 ? make_float2((float)(int8_t)two, (float)(int8_t)(two >> 8)) : decode_e4m3x2(two);
        v[i] = f.x * s, v[i + 1] = f.y * s;
    }
    constexpr int kElem = DT == MOE_F32 ? 4 : 2;
    uint8_t *to = static_cast<uint8_t *>(x) + row * H * kElem;
    if (wide)
        store8<DT, 16>(to, c, 8, v);
    else
        store8<DT, kElem>(to, c, n == 8 ? 8 : n, v);
}

bool aligned(const void *p, uintptr_t n) { return (uintptr_t)p % n == 0; }
uintptr_t size_of(int dt) { return dt == MOE_F32 ? 4 : 2; }
bool is_float(int dt) { return dt == MOE_F16 || dt == MOE_BF16 || dt == MOE_F32; }
mrr_status done()
{
    return cudaGetLastError() == cudaSuccess ? MRR_OK : MRR_ERR_CUDA;
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
    p.q_wide = quant == MOE_Q_MXFP4 ? H % 8 == 0 && aligned(q, 4) : H % 8 == 0 && aligned(q, 8);
    p.eps = eps;
    // what every row's first element is aligned to
    uintptr_t all = (uintptr_t)x | (uintptr_t)weight | (uintptr_t)h | (uintptr_t)y;
    if (T > 1)
        all |= (uintptr_t)x_stride * size | (h || y ? (uintptr_t)H * size : 0);
    if (residual)
        all |= (uintptr_t)residual | (T > 1 ? (uintptr_t)residual_stride * size : 0);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dt == MOE_F32)
        launch<MOE_F32>(p, all, st);
    else if (dt == MOE_BF16)
        launch<MOE_BF16>(p, all, st);
    else
        launch<MOE_F16>(p, all, st);
    return done();
}

mrr_status moe_dequantize_rows_run(const void *q, const void *scales, moe_quant quant, int64_t T, int64_t H,
                                   moe_dtype dt, void *x, mrr_stream_t stream)
{
    if (!is_float(dt))
        return MRR_ERR_DTYPE;
    if (quant < MOE_Q_INT8 || quant > MOE_Q_MXFP8)
        return MRR_ERR_ATTR;
    const int64_t chunks = (H + 7) / 8;
    if (T < 0 || T > INT32_MAX || H < 1 || H > (1 << 20) || T * chunks > 256ll * INT32_MAX)
        return MRR_ERR_SHAPE;
    if (T > 0 && (!q || !scales || !x))
        return MRR_ERR_NULL;
    if (!aligned(x, size_of(dt)) || (quant != MOE_Q_MXFP8 && !aligned(scales, 4)))
        return MRR_ERR_ALIGN;
    if (T == 0)
        return MRR_OK;
    const int wide = H % 8 == 0 && aligned(q, 8) && aligned(x, 16);
    const unsigned grid = (unsigned)((T * chunks + 255) / 256);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    auto kernel = dt == MOE_F32 ? dequantize<MOE_F32> : dt == MOE_BF16 ? dequantize<MOE_BF16> : dequantize<MOE_F16>;
    kernel<<<grid, 256, 0, st>>>(static_cast<const uint8_t *>(q), scales, quant, T, (int)H, (int)chunks, wide, x);
    return done();
}

}  // extern "C"
