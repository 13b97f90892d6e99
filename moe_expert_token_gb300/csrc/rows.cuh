// Eight consecutive elements of a row in registers, e4m3 codes, and sums over a warp or a block.
#pragma once

#include "mx.cuh"

namespace moe_rows {

using namespace moe_mx;

constexpr uint32_t kFull = 0xffffffffu;

// Elements c .. c + n - 1 of a row of DT whose elements c (a multiple of 8) lie at addresses aligned to W bytes,
// as floats; zeros for the others of the 8 (n may be 0 or less, or above 8).
template <int DT, int W>
__device__ __forceinline__ void load8(const void *row, int c, int n, float (&v)[8])
{
    constexpr int kElem = DT == MOE_F32 ? 4 : 2, kWords = 2 * kElem;
    const uint8_t *p = static_cast<const uint8_t *>(row) + (int64_t)c * kElem;
    if (n >= 8) {
        uint32_t w[kWords];
        if constexpr (W == 16) {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p + 4 * i));
                w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
            }
        } else if constexpr (W == 8) {
#pragma unroll
            for (int i = 0; i < kWords; i += 2) {
                const uint2 q = __ldg(reinterpret_cast<const uint2 *>(p + 4 * i));
                w[i] = q.x, w[i + 1] = q.y;
            }
        } else if constexpr (W == 4) {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = __ldg(reinterpret_cast<const uint32_t *>(p + 4 * i));
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = __ldg(reinterpret_cast<const uint16_t *>(p + 4 * i)) |
                       (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(p + 4 * i) + 1) << 16;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if constexpr (DT == MOE_F32) {
                v[i] = __uint_as_float(w[i]);
            } else {
                const float2 f = unpack2<DT>(w[i / 2]);
                v[i] = i % 2 ? f.y : f.x;
            }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = i < n ? load1<DT>(row, c + i) : 0.0f;
    }
}

template <int DT, int W>
__device__ __forceinline__ void store8(void *row, int c, int n, const float (&v)[8])
{
    constexpr int kElem = DT == MOE_F32 ? 4 : 2, kWords = 2 * kElem;
    uint8_t *p = static_cast<uint8_t *>(row) + (int64_t)c * kElem;
    if (n >= 8) {
        uint32_t w[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if constexpr (DT == MOE_F32)
                w[i] = __float_as_uint(v[i]);
            else
                w[i] = pack2<DT>(v[2 * i], v[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if constexpr (W == 16) {
                if (i % 4 == 0)
                    *reinterpret_cast<uint4 *>(p + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
            } else if constexpr (W == 8) {
                if (i % 2 == 0)
                    *reinterpret_cast<uint2 *>(p + 4 * i) = make_uint2(w[i], w[i + 1]);
            } else if constexpr (W == 4) {
                *reinterpret_cast<uint32_t *>(p + 4 * i) = w[i];
            } else {
                reinterpret_cast<uint16_t *>(p + 4 * i)[0] = (uint16_t)w[i];
                reinterpret_cast<uint16_t *>(p + 4 * i)[1] = (uint16_t)(w[i] >> 16);
            }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                store1<DT>(row, c + i, v[i]);
    }
}

// four floats to four e4m3 codes, element 0 in the lowest byte: to nearest, ties to even, held to 448
__device__ __forceinline__ uint32_t encode_e4m3(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// the values of two e4m3 codes (exact in float16)
__device__ __forceinline__ float2 decode_e4m3x2(uint32_t two)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d /= 2)
        v += __shfl_xor_sync(kFull, v, d);
    return v;
}

}  // namespace moe_rows
