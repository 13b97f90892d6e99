// MXFP4 quantisation and its inverse (include/moe_mx.h).
//
// A block of 32 elements shares the scale 2^X, X = floor(log2 max|x|) - 2, and an element becomes
// the e2m1 value nearest to x / 2^X.  Both directions read and write each byte once and compute
// a handful of operations on it, so HBM bounds them.
//
// Layout of the work: a thread owns 8 consecutive elements (one 16-byte load of 16-bit values, one
// 4-byte store of codes), four neighbouring lanes a block, whose maximum takes two shuffles.
#include <type_traits>

#include "mx.cuh"

using namespace moe_mx;

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kFull = 0xffffffffu;

// Eight consecutive elements as they lie in memory (a 16-byte aligned address), their largest
// magnitude as float bits (NaN if one is), and themselves times r.
template <int DT>
struct Chunk {
    uint32_t w[DT == MOE_F32 ? 8 : 4];

    __device__ __forceinline__ void load(const void *x, int64_t i)
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(x) + i * (DT == MOE_F32 ? 4 : 2));
#pragma unroll
        for (int h = 0; h < (DT == MOE_F32 ? 2 : 1); ++h) {
            const uint4 q = __ldg(p + h);
            w[4 * h] = q.x, w[4 * h + 1] = q.y, w[4 * h + 2] = q.z, w[4 * h + 3] = q.w;
        }
    }

    __device__ __forceinline__ uint32_t largest() const
    {
        if constexpr (DT == MOE_F32) {
            uint32_t m = 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                m = max(m, w[j] & 0x7fffffffu);
            return m;
        } else {   // two at a time: unpacking first made this the larger part of the kernel's instructions
            using V = typename std::conditional<DT == MOE_BF16, __nv_bfloat162, __half2>::type;
            auto mag = [&](int j) { return __habs2(*reinterpret_cast<const V *>(&w[j])); };
            const V m = __hmax2_nan(__hmax2_nan(mag(0), mag(1)), __hmax2_nan(mag(2), mag(3)));
            const float2 f = unpack2<DT>(*reinterpret_cast<const uint32_t *>(&m));
            return max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu);
        }
    }

    __device__ __forceinline__ void scaled(float r, float (&v)[8]) const
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = DT == MOE_F32 ? make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[DT == MOE_F32 ? 2 * j + 1 : 0]))
                                           : unpack2<DT>(w[j]);
            v[2 * j] = f.x * r, v[2 * j + 1] = f.y * r;
        }
    }
};

// Rows without gaps (stride K), K a multiple of 64, x and codes aligned for wide accesses: codes
// and scales are then flat arrays too.  A thread takes `kQuantizeChunks` chunks of 8, a block's width
// apart, all loaded before the first is used.
constexpr int kQuantizeChunks = 4;

template <int DT>
__global__ void __launch_bounds__(kThreads) quantize_flat(const void *x, int64_t chunks, uint32_t *codes, uint8_t *scales)
{
    const int64_t c0 = (int64_t)blockIdx.x * (kThreads * kQuantizeChunks) + threadIdx.x;
    Chunk<DT> q[kQuantizeChunks];
#pragma unroll
    for (int u = 0; u < kQuantizeChunks; ++u)
        if (c0 + u * kThreads < chunks)
            q[u].load(x, 8 * (c0 + u * kThreads));
#pragma unroll
    for (int u = 0; u < kQuantizeChunks; ++u) {
        const int64_t c = c0 + u * kThreads;
        if (c >= chunks)   // chunks is a multiple of 8: the lanes of a block agree
            break;
        const uint32_t four = 0xfu << (threadIdx.x % 32 & 28);
        uint32_t m = q[u].largest();
        m = max(m, __shfl_xor_sync(four, m, 1));
        m = max(m, __shfl_xor_sync(four, m, 2));
        const uint32_t s = scale_byte(m);
        float v[8];
        q[u].scaled(inverse_scale(s), v);
        codes[c] = encode8(v);
        if (threadIdx.x % 4 == 0)
            scales[c / 4] = (uint8_t)s;
    }
}

// The inverse: a thread writes 16 bytes (8 elements of 16 bits, 4 of 32) kDequantizeChunks times.
constexpr int kDequantizeChunks = 4;

template <int DT>
__global__ void __launch_bounds__(kThreads) dequantize_flat(const void *codes, const uint8_t *scales, int64_t chunks, void *x)
{
    constexpr int kEach = DT == MOE_F32 ? 4 : 8;
    const int64_t c0 = (int64_t)blockIdx.x * (kThreads * kDequantizeChunks) + threadIdx.x;
    uint32_t q[kDequantizeChunks], s[kDequantizeChunks];
#pragma unroll
    for (int u = 0; u < kDequantizeChunks; ++u) {
        const int64_t c = c0 + u * kThreads;
        if (c < chunks) {
            q[u] = kEach == 8 ? __ldg(static_cast<const uint32_t *>(codes) + c)
                              : (uint32_t)__ldg(static_cast<const uint16_t *>(codes) + c);
            s[u] = __ldg(scales + c / (kBlock / kEach));
        }
    }
#pragma unroll
    for (int u = 0; u < kDequantizeChunks; ++u) {
        const int64_t c = c0 + u * kThreads;
        if (c >= chunks)
            break;
        const float f = e8m0_value(s[u]);
        float v[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            v[j] = decode1(q[u] >> (4 * j)) * f;
        uint4 *to = static_cast<uint4 *>(x) + c;
        if constexpr (kEach == 4)
            *to = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        else
            *to = make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7]));
    }
}

// two neighbouring elements, and back; pair: the address is aligned to both
template <int DT>
__device__ __forceinline__ float2 load2(const void *x, int64_t i, bool pair)
{
    if (pair && DT == MOE_F32)
        return __ldg(reinterpret_cast<const float2 *>(static_cast<const float *>(x) + i));
    if (pair)
        return unpack2<DT>(__ldg(reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(x) + i)));
    return make_float2(load1<DT>(x, i), load1<DT>(x, i + 1));
}

template <int DT>
__device__ __forceinline__ void store2(void *x, int64_t i, float a, float b, bool pair)
{
    if (pair && DT == MOE_F32) {
        *reinterpret_cast<float2 *>(static_cast<float *>(x) + i) = make_float2(a, b);
    } else if (pair) {
        *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(x) + i) = pack2<DT>(a, b);
    } else {
        store1<DT>(x, i, a);
        store1<DT>(x, i + 1, b);
    }
}

// Any even K, any stride and alignment: a lane has two elements of a block pair (64 elements), a warp
// kPairs of them in a row, all loaded before the first is used.
constexpr int kPairs = 8;

template <int DT>
__global__ void __launch_bounds__(kThreads) quantize_any(const void *x, int64_t K, int64_t stride, int64_t runs,
                                                         int64_t units, bool pair, uint8_t *codes, uint8_t *scales)
{
    const int lane = threadIdx.x % 32;
    const int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32, pairs = (K + 63) / 64;
    if (u >= units)
        return;
    const int64_t row = u / runs, p0 = (u - row * runs) * kPairs, k0 = p0 * 64 + 2 * lane;
    float2 v[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i)   // K is even: both elements or none
        v[i] = k0 + 64 * i < K ? load2<DT>(x, row * stride + k0 + 64 * i, pair) : make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        if (p0 + i >= pairs)
            break;
        const bool in = k0 + 64 * i < K;
        uint32_t m = max(__float_as_uint(v[i].x) & 0x7fffffffu, __float_as_uint(v[i].y) & 0x7fffffffu);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            m = max(m, __shfl_xor_sync(kFull, m, o));
        const uint32_t s = scale_byte(m);
        const float r = inverse_scale(s);
        if (in)
            codes[row * (K / 2) + k0 / 2 + 32 * i] = (uint8_t)encode2(v[i].x * r, v[i].y * r);
        if (lane % 16 == 0)
            scales[(row * pairs + p0 + i) * 2 + lane / 16] = (uint8_t)(in ? s : 127u);   // a second block past K: 127
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) dequantize_any(const uint8_t *codes, const uint8_t *scales, int64_t K,
                                                           int64_t stride, int64_t runs, int64_t units, bool pair, void *x)
{
    const int lane = threadIdx.x % 32;
    const int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32, pairs = (K + 63) / 64;
    if (u >= units)
        return;
    const int64_t row = u / runs, p0 = (u - row * runs) * kPairs, k0 = p0 * 64 + 2 * lane;
    uint32_t q[kPairs], s[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
        if (k0 + 64 * i < K) {
            q[i] = __ldg(codes + row * (K / 2) + k0 / 2 + 32 * i);
            s[i] = __ldg(scales + (row * pairs + p0 + i) * 2 + lane / 16);
        }
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
        if (k0 + 64 * i < K) {
            const float f = e8m0_value(s[i]);
            store2<DT>(x, row * stride + k0 + 64 * i, decode1(q[i]) * f, decode1(q[i] >> 4) * f, pair);
        }
}

mrr_status check(const void *x, moe_dtype dt, int64_t rows, int64_t K, int64_t stride, const void *codes,
                 const void *scales)
{
    if (dt != MOE_F16 && dt != MOE_BF16 && dt != MOE_F32)
        return MRR_ERR_DTYPE;
    if (rows < 0 || rows > INT32_MAX || K < 2 || K % 2 || K > (int64_t(1) << 30) || rows * ((K + 511) / 512) > INT32_MAX ||
        stride < K ||
        stride > (int64_t(1) << 31))
        return MRR_ERR_SHAPE;
    if (rows > 0 && (!x || !codes || !scales))
        return MRR_ERR_NULL;
    if ((uintptr_t)x % (dt == MOE_F32 ? 4 : 2))
        return MRR_ERR_ALIGN;
    return MRR_OK;
}

// the flat kernels' conditions (codes are read and written in 4-byte words)
bool flat(const void *x, int64_t K, int64_t stride, const void *codes)
{
    return K % 64 == 0 && stride == K && (uintptr_t)x % 16 == 0 && (uintptr_t)codes % 4 == 0;
}

// the general kernels' launch
struct Shape {
    int64_t runs, units;   // runs of kPairs block pairs in a row, and in all rows
    unsigned grid;
    bool pair;             // two elements can be loaded and stored at once
    Shape(const void *x, int64_t rows, int64_t K, int64_t stride, int dt)
    {
        runs = ((K + 63) / 64 + kPairs - 1) / kPairs;
        units = rows * runs;
        grid = (unsigned)((units + kThreads / 32 - 1) / (kThreads / 32));
        pair = stride % 2 == 0 && (uintptr_t)x % (dt == MOE_F32 ? 8 : 4) == 0;
    }
};

template <int DT>
void launch_quantize(const void *x, int64_t rows, int64_t K, int64_t stride, uint8_t *codes, uint8_t *scales,
                     cudaStream_t st)
{
    if (flat(x, K, stride, codes)) {
        const int64_t chunks = rows * (K / 8), per = kThreads * kQuantizeChunks;
        quantize_flat<DT><<<(unsigned)((chunks + per - 1) / per), kThreads, 0, st>>>(
            x, chunks, reinterpret_cast<uint32_t *>(codes), scales);
        return;
    }
    const Shape s(x, rows, K, stride, DT);
    quantize_any<DT><<<s.grid, kThreads, 0, st>>>(x, K, stride, s.runs, s.units, s.pair, codes, scales);
}

template <int DT>
void launch_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t K, void *x, int64_t stride,
                       cudaStream_t st)
{
    if (flat(x, K, stride, codes)) {
        const int64_t chunks = rows * (K / (DT == MOE_F32 ? 4 : 8)), per = kThreads * kDequantizeChunks;
        dequantize_flat<DT><<<(unsigned)((chunks + per - 1) / per), kThreads, 0, st>>>(codes, scales, chunks, x);
        return;
    }
    const Shape s(x, rows, K, stride, DT);
    dequantize_any<DT><<<s.grid, kThreads, 0, st>>>(codes, scales, K, stride, s.runs, s.units, s.pair, x);
}

}  // namespace

extern "C" {

mrr_status moe_mx_quantize_run(const void *x, moe_dtype dt, int64_t rows, int64_t K, int64_t row_stride,
                               uint8_t *codes, uint8_t *scales, mrr_stream_t stream)
{
    const mrr_status st = check(x, dt, rows, K, row_stride, codes, scales);
    if (st != MRR_OK || rows == 0)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dt == MOE_F32)
        launch_quantize<MOE_F32>(x, rows, K, row_stride, codes, scales, s);
    else if (dt == MOE_BF16)
        launch_quantize<MOE_BF16>(x, rows, K, row_stride, codes, scales, s);
    else
        launch_quantize<MOE_F16>(x, rows, K, row_stride, codes, scales, s);
    return cudaGetLastError() == cudaSuccess ? MRR_OK : MRR_ERR_CUDA;
}

mrr_status moe_mx_dequantize_run(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t K, moe_dtype dt,
                                 void *x, int64_t row_stride, mrr_stream_t stream)
{
    const mrr_status st = check(x, dt, rows, K, row_stride, codes, scales);
    if (st != MRR_OK || rows == 0)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dt == MOE_F32)
        launch_dequantize<MOE_F32>(codes, scales, rows, K, x, row_stride, s);
    else if (dt == MOE_BF16)
        launch_dequantize<MOE_BF16>(codes, scales, rows, K, x, row_stride, s);
    else
        launch_dequantize<MOE_F16>(codes, scales, rows, K, x, row_stride, s);
    return cudaGetLastError() == cudaSuccess ? MRR_OK : MRR_ERR_CUDA;
}

}  // extern "C"
