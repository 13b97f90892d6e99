// MXFP4 quantisation and its inverse (include/moe_mx.h).
//
// A block of 32 elements shares the scale 2^X, X = floor(log2 max|x|) - 2, and an element becomes
// the e2m1 value nearest to x / 2^X.  Both directions read and write each byte once and compute
// a handful of operations on it, so HBM bounds them.
//
// Layout of the work: a thread owns 8 consecutive elements (one 16-byte load of 16-bit values, one
// 4-byte store of codes), four neighbouring lanes a block, whose maximum takes two shuffles.
#include "mx.cuh"

using namespace moe_mx;

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr uint32_t kFull = 0xffffffffu;

// eight consecutive elements at x + i; the address is 16-byte aligned
template <int DT>
__device__ __forceinline__ void load8(const void *x, int64_t i, float (&v)[8])
{
    if (DT == MOE_F32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + i));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = unpack2<DT>(w[j]);
            v[2 * j] = f.x, v[2 * j + 1] = f.y;
        }
    }
}

template <int DT>
__device__ __forceinline__ void store8(void *x, int64_t i, const float (&v)[8])
{
    if (DT == MOE_F32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(x) + i);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(x) + i) =
            make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7]));
    }
}

// Rows without gaps (stride K), K a multiple of 64, x and codes aligned for wide accesses: codes
// and scales are then flat arrays too, and a thread takes kUnroll chunks of 8, a block's width
// apart, all loaded before the first is used.
template <int DT>
__global__ void __launch_bounds__(kThreads) quantize_flat(const void *x, int64_t chunks, uint32_t *codes, uint8_t *scales)
{
    const int64_t c0 = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
    float v[kUnroll][8];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        if (c0 + u * kThreads < chunks)
            load8<DT>(x, 8 * (c0 + u * kThreads), v[u]);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t c = c0 + u * kThreads;
        if (c >= chunks)   // chunks is a multiple of 8: the lanes of a block agree
            break;
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            m = max(m, __float_as_uint(v[u][j]) & 0x7fffffffu);
        const uint32_t four = 0xfu << (threadIdx.x % 32 & 28);
        m = max(m, __shfl_xor_sync(four, m, 1));
        m = max(m, __shfl_xor_sync(four, m, 2));
        const uint32_t s = scale_byte(m);
        const float r = inverse_scale(s);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[u][j] *= r;
        codes[c] = encode8(v[u]);
        if (threadIdx.x % 4 == 0)
            scales[c / 4] = (uint8_t)s;
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) dequantize_flat(const uint32_t *codes, const uint8_t *scales, int64_t chunks,
                                                            void *x)
{
    const int64_t c0 = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
    uint32_t q[kUnroll], s[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t c = c0 + u * kThreads;
        if (c < chunks) {
            q[u] = __ldg(codes + c);
            s[u] = __ldg(scales + c / 4);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t c = c0 + u * kThreads;
        if (c >= chunks)
            break;
        float v[8];
        decode8(q[u], v);
        const float f = e8m0_value(s[u]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] *= f;
        store8<DT>(x, 8 * c, v);
    }
}

// Any even K, any stride and alignment: one warp per block pair (64 elements), two elements a lane.
template <int DT>
__global__ void __launch_bounds__(kThreads) quantize_any(const void *x, int64_t rows, int64_t K, int64_t stride,
                                                         uint8_t *codes, uint8_t *scales)
{
    const int64_t pairs = (K + 63) / 64;
    const int lane = threadIdx.x % 32;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; u < rows * pairs; u += warps) {
        const int64_t row = u / pairs, k = (u - row * pairs) * 64 + 2 * lane;
        const bool in = k < K;   // K is even: both elements or none
        const float a = in ? load1<DT>(x, row * stride + k) : 0.f, b = in ? load1<DT>(x, row * stride + k + 1) : 0.f;
        uint32_t m = max(__float_as_uint(a) & 0x7fffffffu, __float_as_uint(b) & 0x7fffffffu);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            m = max(m, __shfl_xor_sync(kFull, m, o));
        const uint32_t s = scale_byte(m);
        const float r = inverse_scale(s);
        if (in)
            codes[row * (K / 2) + k / 2] = (uint8_t)encode2(a * r, b * r);
        if (lane % 16 == 0)
            scales[u * 2 + lane / 16] = (uint8_t)(in ? s : 127u);   // a second block past K: 127
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) dequantize_any(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                                           int64_t K, void *x, int64_t stride)
{
    const int64_t pairs = (K + 63) / 64;
    const int lane = threadIdx.x % 32;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; u < rows * pairs; u += warps) {
        const int64_t row = u / pairs, k = (u - row * pairs) * 64 + 2 * lane;
        if (k >= K)
            continue;
        const uint32_t q = __ldg(codes + row * (K / 2) + k / 2);
        const float s = e8m0_value(__ldg(scales + u * 2 + lane / 16));
        store1<DT>(x, row * stride + k, decode1(q) * s);
        store1<DT>(x, row * stride + k + 1, decode1(q >> 4) * s);
    }
}

mrr_status check(const void *x, moe_dtype dt, int64_t rows, int64_t K, int64_t stride, const void *codes,
                 const void *scales)
{
    if (dt != MOE_F16 && dt != MOE_BF16 && dt != MOE_F32)
        return MRR_ERR_DTYPE;
    if (rows < 0 || rows > INT32_MAX || K < 2 || K % 2 || K > (int64_t(1) << 30) || stride < K ||
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

template <int DT>
void launch_quantize(const void *x, int64_t rows, int64_t K, int64_t stride, uint8_t *codes, uint8_t *scales,
                     cudaStream_t st)
{
    if (flat(x, K, stride, codes)) {
        const int64_t chunks = rows * (K / 8), per = kThreads * kUnroll;
        quantize_flat<DT><<<(unsigned)((chunks + per - 1) / per), kThreads, 0, st>>>(
            x, chunks, reinterpret_cast<uint32_t *>(codes), scales);
        return;
    }
    const int64_t warps = rows * ((K + 63) / 64);
    const int64_t grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
    quantize_any<DT><<<(unsigned)(grid < 65535 * 16 ? grid : 65535 * 16), kThreads, 0, st>>>(x, rows, K, stride, codes,
                                                                                            scales);
}

template <int DT>
void launch_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t K, void *x, int64_t stride,
                       cudaStream_t st)
{
    if (flat(x, K, stride, codes)) {
        const int64_t chunks = rows * (K / 8), per = kThreads * kUnroll;
        dequantize_flat<DT><<<(unsigned)((chunks + per - 1) / per), kThreads, 0, st>>>(
            reinterpret_cast<const uint32_t *>(codes), scales, chunks, x);
        return;
    }
    const int64_t warps = rows * ((K + 63) / 64);
    const int64_t grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
    dequantize_any<DT><<<(unsigned)(grid < 65535 * 16 ? grid : 65535 * 16), kThreads, 0, st>>>(codes, scales, rows, K,
                                                                                              x, stride);
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
