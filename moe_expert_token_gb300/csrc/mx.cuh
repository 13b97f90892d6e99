// MXFP4 in registers: e2m1 codes, e8m0 scales, and loads / stores of the row types beside them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_mx.h"

namespace moe_mx {

constexpr int kBlock = 32;   // elements of one scale

__host__ __device__ constexpr int64_t scale_row_bytes(int64_t K) { return (K + 63) / 64 * 2; }

// 2^(b - 127); 255 is NaN and 0 the subnormal 2^-127
__device__ __forceinline__ float e8m0_value(uint32_t b)
{
    const uint32_t bits = b == 0u ? 0x00400000u : (b == 255u ? 0x7fffffffu : b << 23);
    return __uint_as_float(bits);
}

// The scale byte of a block whose largest magnitude has the float bits `amax` (sign clear):
// 2^(floor(log2 m) - 2).  The exponent field of a normal m is floor(log2 m) + 127, so the byte is
// that field less 2, held to 0 from below (2^-127; a subnormal m has field 0 and lands there too).
// A NaN or infinity gives 255.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax)
{
    const uint32_t field = amax >> 23;
    return field == 255u ? 255u : (field > 2u ? field - 2u : 0u);
}

// 1 / 2^(b - 127) for b <= 252, the largest byte a finite block gets: 2^(127 - b), normal from
// 2^-125 to 2^127
__device__ __forceinline__ float inverse_scale(uint32_t b) { return __uint_as_float((254u - min(b, 252u)) << 23); }

// eight floats (already divided by the scale) to eight codes, element 0 in the lowest four bits;
// the conversion rounds to nearest, ties to even, and saturates at 6
__device__ __forceinline__ uint32_t encode8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The value of a code (its low four bits): magnitude bits e e m over a bias of 1 are a float's
// exponent and mantissa head; as a float with those bits the value is 2^-126 times too small
// (0.5 is then subnormal), which the product puts right exactly.
__device__ __forceinline__ float decode1(uint32_t code)
{
    const float tiny = __uint_as_float(((code & 8u) << 28) | ((code & 7u) << 22));
    return tiny * 0x1p126f;
}

__device__ __forceinline__ void decode8(uint32_t w, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = decode1(w >> (4 * i));
}

template <int DT>
__device__ __forceinline__ float load1(const void *p, int64_t i)
{
    if (DT == MOE_F32)
        return __ldg(static_cast<const float *>(p) + i);
    if (DT == MOE_BF16)
        return __bfloat162float(__ldg(static_cast<const __nv_bfloat16 *>(p) + i));
    return __half2float(__ldg(static_cast<const __half *>(p) + i));
}

template <int DT>
__device__ __forceinline__ void store1(void *p, int64_t i, float v)
{
    if (DT == MOE_F32)
        static_cast<float *>(p)[i] = v;
    else if (DT == MOE_BF16)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(p)[i] = __float2half_rn(v);
}

// two 16-bit values of one word, and back
template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t w)
{
    if (DT == MOE_BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if (DT == MOE_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

}  // namespace moe_mx
