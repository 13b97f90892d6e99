// A residual's addition and the root-mean-square norm of the sum, with its 8-bit and MXFP4 forms (include/moe_norm.h).
//
// h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight: every element is read and written once and a
// handful of operations are made of it, so HBM bounds both.  A row stays in registers, 8 elements a
// chunk, between the sum of its squares and the results: it belongs to one block (or, where it is short,
// to one warp).
#pragma once

#include "moe_norm.h"
#include "rms_norm.h"
#include "rows.cuh"

namespace moe_norm {
namespace {

using namespace moe_rows;

constexpr int kMaxWarps = 32;

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

// y / s, rounded once: y times the rounded reciprocal, and Markstein's correction by what that leaves of y (two operations, 0.2 us
// of 154).  It is right where the remainder is exact: see widen.
__device__ __forceinline__ float over(float y, float s, float inverse)
{
    const float q = y * inverse;
    return fmaf(fmaf(-q, s, y), inverse, q);
}

// The remainder is a multiple of the quotient's last place times s's, and passes out of float32 under scales of about 2^-100.
// So y and s are taken 2^64 times as large where s is below 2^-64, which is exact (quotients that give a code other than 0
// are 2^-11 or more).  In a branch, which rows hardly ever take (16384 x 7172 int8: 167 us, 166 without; 65536 x 512: 54 and 54,
// e4m3_128 67 and 65); as a factor in every quotient it is registers: 184 and 60 us.
__device__ __forceinline__ void widen(float (&y)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        y[j] *= 0x1p64f;
}

__device__ __forceinline__ bool widen_scale(float &s, float &inverse)
{
    if (s >= 0x1p-64f || s != s)
        return false;
    s *= 0x1p64f;
    inverse *= 0x1p-64f;
    return true;
}

__device__ __forceinline__ uint32_t int8_of(float v) { return (uint32_t)min(127, max(-127, __float2int_rn(v))) & 0xffu; }

// BYTES (4 or 8) bytes of codes, of which the row has n, in stores as wide as their place allows
template <int BYTES>
__device__ __forceinline__ void store_codes(uint8_t *to, int n, int align, uint32_t lo, uint32_t hi)
{
    if (n >= BYTES && align >= 4) {
        if (BYTES == 8 && align == 8) {
            *reinterpret_cast<uint2 *>(to) = make_uint2(lo, hi);
        } else {
            *reinterpret_cast<uint32_t *>(to) = lo;
            if (BYTES == 8)
                *reinterpret_cast<uint32_t *>(to + 4) = hi;
        }
    } else if (n >= BYTES && align == 2) {
#pragma unroll
        for (int i = 0; i < BYTES; i += 2)
            *reinterpret_cast<uint16_t *>(to + i) = (uint16_t)((i < 4 ? lo : hi) >> (8 * (i % 4)));
    } else {
#pragma unroll
        for (int i = 0; i < BYTES; ++i)
            if (i < n)
                to[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i % 4)));
    }
}

// codes of a chunk (elements c .. c + n - 1 of row `row`), from their values over the scale
__device__ __forceinline__ void store_bytes(const Params &p, int64_t row, int c, int n, uint32_t lo, uint32_t hi)
{
    store_codes<8>(static_cast<uint8_t *>(p.q) + row * p.H + c, n, p.q_align, lo, hi);
}

__device__ __forceinline__ uint32_t largest(const float (&v)[8])
{
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

// y's chunks of one row to codes and scales; y is used up.  A block of 32 elements is 4 lanes' chunks, one of 128 elements 16 lanes'.
template <int NV, bool kBlock>
__device__ __forceinline__ void quantize(const Params &p, int64_t row, int tid, int threads, float (&y)[NV][8],
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
        float s = float_scale(m, kind == MOE_Q_INT8 ? 127.0f : 448.0f, inverse);
        if (tid == 0)
            static_cast<float *>(p.scales)[row] = s;
        if (widen_scale(s, inverse)) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                widen(y[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (tid + i * threads), n = p.H - c;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = over(y[i][j], s, inverse);
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
        float inverse, s = 0.0f;
        if (kind == MOE_Q_E4M3_128) {
            m = max(m, __shfl_xor_sync(kFull, m, 4));
            m = max(m, __shfl_xor_sync(kFull, m, 8));
            s = float_scale(m, 448.0f, inverse);
            if (c % 128 == 0 && n > 0)
                static_cast<float *>(p.scales)[row * ((p.H + 127) / 128) + c / 128] = s;
            if (widen_scale(s, inverse))
                widen(y[i]);
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
            v[j] = kind == MOE_Q_E4M3_128 ? over(y[i][j], s, inverse) : y[i][j] * inverse;   // (by a power of two: exact)
        if (kind == MOE_Q_MXFP4) {
            store_codes<4>(static_cast<uint8_t *>(p.q) + (row * p.H + c) / 2, n / 2, p.q_align, encode8(v), 0u);
        } else {
            store_bytes(p, row, c, n, encode_e4m3(v[0], v[1], v[2], v[3]), encode_e4m3(v[4], v[5], v[6], v[7]));
        }
    }
}

// NV chunks a thread; kBlock: a block has a row, else each of its warps has one.  (Warps with 4 chunks of 16-bit rows: four
// blocks an SM, 64 registers; with 67 they are three and 65536 x 512 int8 takes 60 us instead of 54.)
template <int DT, int W, int NV, bool kBlock>
__global__ void __launch_bounds__(kBlock ? 1024 : 256, !kBlock && W == 16 && NV == 4 && DT != MOE_F32 ? 4 : 0) add_rms_norm(Params p)
{
    __shared__ float sums[kMaxWarps];
    __shared__ uint32_t tops[kMaxWarps];
    const int threads = kBlock ? blockDim.x : 32, tid = kBlock ? threadIdx.x : threadIdx.x % 32;
    const int64_t row = kBlock ? blockIdx.x : (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    if (row >= p.T)
        return;
    using C = Chunk<DT, W>;
    const int size = p.H * C::kElem;   // of a row, in bytes
    const uint8_t *x = static_cast<const uint8_t *>(p.x) + row * p.x_stride * C::kElem;
    const uint8_t *res = static_cast<const uint8_t *>(p.residual) + row * p.residual_stride * C::kElem;
    float v[NV][8], w[8];
    {
        C a[NV], b[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            a[i].load(x, (tid + i * threads) * C::kBytes, size);
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                b[i].load(res, (tid + i * threads) * C::kBytes, size);
        }
        if (NV == 1)   // few rows: nothing else hides the weight's latency
            load_weight<DT, W>(p.weight, p.weight_f32, tid, p.H, w);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            a[i].get(v[i]);
            if (p.residual) {
                float r[8];
                b[i].get(r);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i][j] += r[j];
            }
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum = fmaf(v[i][j], v[i][j], sum);
        if (p.h) {
            C out;
            out.set(v[i]);
            out.store(static_cast<uint8_t *>(p.h) + row * size, (tid + i * threads) * C::kBytes, size);
        }
    }
    sum = row_sum<kBlock>(sum, sums);
    const float r = 1.0f / sqrtf(sum / (float)p.H + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (NV > 1)
            load_weight<DT, W>(p.weight, p.weight_f32, tid + i * threads, p.H, w);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[i][j] = v[i][j] * r * w[j];
        if (p.y) {
            C out;
            out.set(v[i]);
            out.store(static_cast<uint8_t *>(p.y) + row * size, (tid + i * threads) * C::kBytes, size);
        }
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
    // Few rows: as many threads to a row as there are chunks.  Many: two or four chunks a thread.
    auto threads = [&](int each) { return (unsigned)(((chunks + each - 1) / each + 31) / 32 * 32); };
    const unsigned grid = (unsigned)p.T;
    if (p.T <= 304 && chunks <= 1024)
        add_rms_norm<DT, W, 1, true><<<grid, threads(1), 0, st>>>(p);
    else if (chunks <= 512)
        add_rms_norm<DT, W, 2, true><<<grid, threads(2), 0, st>>>(p);
    else if (chunks <= 4096)
        add_rms_norm<DT, W, 4, true><<<grid, threads(4), 0, st>>>(p);
    else
        add_rms_norm<DT, W, 8, true><<<grid, threads(8), 0, st>>>(p);
}

template <int DT>
cudaError_t launch_any(const Params &p, uintptr_t all, cudaStream_t st)
{
    if (all % 16 == 0)
        launch<DT, 16>(p, st);
    else if (all % 8 == 0)
        launch<DT, 8>(p, st);
    else if (all % 4 == 0 || DT == MOE_F32)
        launch<DT, 4>(p, st);
    else
        launch<DT, DT == MOE_F32 ? 4 : 2>(p, st);
    return cudaGetLastError();
}

}  // namespace
}  // namespace moe_norm
