// Eight consecutive elements of a row in registers, e4m3 codes, and sums over a warp or a block.
#pragma once

#include "mx.cuh"

namespace moe_rows {

using namespace moe_mx;

constexpr uint32_t kFull = 0xffffffffu;

// Eight consecutive elements of DT as they lie in a row whose bytes, from its start, come in pieces of W (the row's
// size is a multiple of W, its address aligned to W).  Pieces past the row's end are zeros and are not stored.  A piece
// is loaded under a predicate of its own and without a branch: several chunks' loads are under way at once.
template <int DT, int W>
struct Chunk {
    static constexpr int kElem = DT == MOE_F32 ? 4 : 2, kBytes = 8 * kElem, kWords = kBytes / 4;
    uint32_t w[kWords];

    // bytes at .. at + kBytes - 1 of a row of `size` bytes
    __device__ __forceinline__ void load(const void *row, int at, int size)
    {
        const uint8_t *p = static_cast<const uint8_t *>(row) + at;
#pragma unroll
        for (int i = 0; i < kBytes; i += W) {
            const bool in = at + i < size;
            if constexpr (W == 16) {
                uint4 q = make_uint4(0u, 0u, 0u, 0u);
                if (in)
                    q = __ldg(reinterpret_cast<const uint4 *>(p + i));
                w[i / 4] = q.x, w[i / 4 + 1] = q.y, w[i / 4 + 2] = q.z, w[i / 4 + 3] = q.w;
            } else if constexpr (W == 8) {
                uint2 q = make_uint2(0u, 0u);
                if (in)
                    q = __ldg(reinterpret_cast<const uint2 *>(p + i));
                w[i / 4] = q.x, w[i / 4 + 1] = q.y;
            } else if constexpr (W == 4) {
                w[i / 4] = in ? __ldg(reinterpret_cast<const uint32_t *>(p + i)) : 0u;
            } else {
                const uint32_t half = in ? __ldg(reinterpret_cast<const uint16_t *>(p + i)) : 0u;
                w[i / 4] = i % 4 == 0 ? half : w[i / 4] | half << 16;
            }
        }
    }

    __device__ __forceinline__ void store(void *row, int at, int size) const
    {
        uint8_t *p = static_cast<uint8_t *>(row) + at;
#pragma unroll
        for (int i = 0; i < kBytes; i += W) {
            if (at + i >= size)
                continue;
            if constexpr (W == 16)
                *reinterpret_cast<uint4 *>(p + i) = make_uint4(w[i / 4], w[i / 4 + 1], w[i / 4 + 2], w[i / 4 + 3]);
            else if constexpr (W == 8)
                *reinterpret_cast<uint2 *>(p + i) = make_uint2(w[i / 4], w[i / 4 + 1]);
            else if constexpr (W == 4)
                *reinterpret_cast<uint32_t *>(p + i) = w[i / 4];
            else
                *reinterpret_cast<uint16_t *>(p + i) = (uint16_t)(w[i / 4] >> (i % 4 * 8));
        }
    }

    __device__ __forceinline__ void get(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if constexpr (DT == MOE_F32) {
                v[i] = __uint_as_float(w[i]);
            } else {
                const float2 f = unpack2<DT>(w[i / 2]);
                v[i] = i % 2 ? f.y : f.x;
            }
    }

    __device__ __forceinline__ void set(const float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if constexpr (DT == MOE_F32)
                w[i] = __float_as_uint(v[i]);
            else
                w[i] = pack2<DT>(v[2 * i], v[2 * i + 1]);
    }
};

// chunk c of a norm's weight, which is of DT or float32, as floats
template <int DT, int W>
__device__ __forceinline__ void load_weight(const void *weight, bool is_f32, int c, int H, float (&v)[8])
{
    if (DT == MOE_F32 || is_f32) {
        Chunk<MOE_F32, W == 2 ? 4 : W> w;
        w.load(weight, 32 * c, 4 * H);
        w.get(v);
    } else {
        Chunk<DT, W> w;
        w.load(weight, Chunk<DT, W>::kBytes * c, Chunk<DT, W>::kElem * H);
        w.get(v);
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

// elements first .. first + count - 1 of ELEM bytes (2 or 4; 1: bytes) at `base` to zero, by threads 0 .. threads - 1:
// 16 bytes at a time between the first and last 16-byte boundary
template <int ELEM>
__device__ __forceinline__ void clear(void *base, int64_t first, int64_t count, int thread, int threads)
{
    uint8_t *lo = static_cast<uint8_t *>(base) + first * ELEM, *hi = lo + count * ELEM;
    uint8_t *from = reinterpret_cast<uint8_t *>(((uintptr_t)lo + 15) / 16 * 16);
    uint8_t *to = reinterpret_cast<uint8_t *>((uintptr_t)hi / 16 * 16);
    if (from >= to)
        from = to = hi;
    auto edge = [](uint8_t *q) {
        if constexpr (ELEM == 4)
            *reinterpret_cast<uint32_t *>(q) = 0u;
        else if constexpr (ELEM == 2)
            *reinterpret_cast<uint16_t *>(q) = 0u;
        else
            *q = 0u;
    };
    for (uint8_t *q = lo + (int64_t)ELEM * thread; q < from; q += ELEM * threads)
        edge(q);
    for (uint8_t *q = from + (int64_t)16 * thread; q < to; q += 16 * threads)
        *reinterpret_cast<uint4 *>(q) = make_uint4(0u, 0u, 0u, 0u);
    for (uint8_t *q = to + (int64_t)ELEM * thread; q < hi; q += ELEM * threads)
        edge(q);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d /= 2)
        v += __shfl_xor_sync(kFull, v, d);
    return v;
}

}  // namespace moe_rows
