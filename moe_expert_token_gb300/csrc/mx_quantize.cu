// MXFP4 quantisation and its inverse (include/moe_mx.h).
//
// A block of 32 elements shares the scale 2^X, X = floor(log2 max|x|) - 2, and an element becomes
// the e2m1 value nearest to x / 2^X.  Both directions read and write each byte once and compute
// a handful of operations on it, so HBM bounds them: 16384 x 7168 in bfloat16, 297 MB, take 45.1 us
// (6.6 TB/s) one way and 47.2 us (6.3 TB/s) the other.
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

    // elements i .. i + n - 1 (n up to 8) from an address aligned to W bytes, zeros for the others
    template <int W>
    __device__ __forceinline__ void load(const void *x, int64_t i, int n)
    {
        constexpr int kWords = DT == MOE_F32 ? 8 : 4;
        const uint8_t *p = static_cast<const uint8_t *>(x) + i * (DT == MOE_F32 ? 4 : 2);
        if (W >= 4 && n == 8) {
#pragma unroll
            for (int h = 0; h < kWords; h += W / 4)
                if constexpr (W == 16) {
                    const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p + 4 * h));
                    w[h] = q.x, w[h + 1] = q.y, w[h + 2] = q.z, w[h + 3] = q.w;
                } else if constexpr (W == 8) {
                    const uint2 q = __ldg(reinterpret_cast<const uint2 *>(p + 4 * h));
                    w[h] = q.x, w[h + 1] = q.y;
                } else {
                    w[h] = __ldg(reinterpret_cast<const uint32_t *>(p + 4 * h));
                }
        } else {
#pragma unroll
            for (int h = 0; h < kWords; ++h) {
                w[h] = 0u;
                if constexpr (DT == MOE_F32) {
                    if (h < n)
                        w[h] = __ldg(reinterpret_cast<const uint32_t *>(p) + h);
                } else if (2 * h < n) {   // n is even
                    const uint16_t *e = reinterpret_cast<const uint16_t *>(p) + 2 * h;
                    w[h] = __ldg(e) | (uint32_t)__ldg(e + 1) << 16;
                }
            }
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
// apart, all loaded before the first is used (1, 2 or 8 chunks were slower).
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

// Any even K, any stride and alignment (of x's rows to W bytes, of the codes' to `align`): as above, a lane
// has 8 elements of each chunk, but a warp stays in one row, of which it has run_of() elements, 2 KB.
// It is bound by instructions more than by HBM, so indices inside a row have 32 bits: 16384 x 7152 in
// bfloat16 takes 57 us (5.2 TB/s); with 64-bit indices 62, and 1 KB a warp 69.
template <int DT>
__host__ __device__ constexpr int run_of() { return DT == MOE_F32 ? 512 : 1024; }

// n / 2 bytes of codes (n elements, 8 or fewer; to load: kMost), at an address aligned to `align` bytes
__device__ __forceinline__ void store_codes(uint8_t *to, uint32_t w, int n, int align)
{
    if (n == 8 && align == 4) {
        *reinterpret_cast<uint32_t *>(to) = w;
    } else if (n == 8 && align == 2) {
        reinterpret_cast<uint16_t *>(to)[0] = (uint16_t)w;
        reinterpret_cast<uint16_t *>(to)[1] = (uint16_t)(w >> 16);
    } else {
#pragma unroll
        for (int b = 0; b < 4; ++b)
            if (2 * b < n)
                to[b] = (uint8_t)(w >> (8 * b));
    }
}

template <int kMost>
__device__ __forceinline__ uint32_t load_codes(const uint8_t *from, int n, int align)
{
    if (n == kMost && align >= kMost / 2)
        return kMost == 8 ? __ldg(reinterpret_cast<const uint32_t *>(from)) : (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(from));
    if (n == kMost && align == 2)
        return __ldg(reinterpret_cast<const uint16_t *>(from)) | (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(from) + 1) << 16;
    uint32_t w = 0u;
#pragma unroll
    for (int b = 0; b < kMost / 2; ++b)
        if (2 * b < n)
            w |= (uint32_t)__ldg(from + b) << (8 * b);
    return w;
}

template <int DT, int W>
__global__ void __launch_bounds__(kThreads) quantize_any(const void *x, int K, int64_t stride, uint32_t runs,
                                                         uint32_t units, int align, uint8_t *codes, uint8_t *scales)
{
    const int lane = threadIdx.x % 32;
    const uint32_t u = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    if (u >= units)
        return;
    const int64_t row = u / runs;
    const int first = (int)(u % runs) * run_of<DT>(), blocks = (K + 63) / 64 * 2;
    constexpr int kChunks = run_of<DT>() / 256;
    codes += row * (K / 2);
    scales += row * blocks;
    Chunk<DT> q[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int k = first + 256 * i + 8 * lane;
        q[i].template load<W>(x, row * stride + k, max(0, min(8, K - k)));
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int k = first + 256 * i + 8 * lane;
        uint32_t m = q[i].largest();
        m = max(m, __shfl_xor_sync(kFull, m, 1));
        m = max(m, __shfl_xor_sync(kFull, m, 2));
        const uint32_t s = scale_byte(m);
        float v[8];
        q[i].scaled(inverse_scale(s), v);
        const uint32_t w = encode8(v);
        if (k < K)
            store_codes(codes + k / 2, w, min(8, K - k), align);
        if (lane % 4 == 0 && k / kBlock < blocks)   // a second block past K: 127
            scales[k / kBlock] = (uint8_t)(k < K ? s : 127u);
    }
}

template <int DT, int W>
__global__ void __launch_bounds__(kThreads) dequantize_any(const uint8_t *codes, const uint8_t *scales, int K,
                                                           int64_t stride, uint32_t runs, uint32_t units, int align, void *x)
{
    const int lane = threadIdx.x % 32;
    const uint32_t u = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    if (u >= units)
        return;
    const int64_t row = u / runs;
    const int first = (int)(u % runs) * run_of<DT>(), blocks = (K + 63) / 64 * 2;
    constexpr int kEach = DT == MOE_F32 ? 4 : 8, kChunks = 4;   // 16 bytes of x, as above
    static_assert(kChunks * 32 * kEach == run_of<DT>(), "");
    codes += row * (K / 2);
    scales += row * blocks;
    uint32_t q[kChunks], s[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int k = first + kEach * (32 * i + lane);
        if (k < K) {
            q[i] = load_codes<kEach>(codes + k / 2, min(kEach, K - k), align);
            s[i] = __ldg(scales + k / kBlock);
        }
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int k = first + kEach * (32 * i + lane);
        if (k >= K)
            break;
        const float f = e8m0_value(s[i]);
        float v[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            v[j] = decode1(q[i] >> (4 * j)) * f;
        if (W >= 4 && K - k >= kEach) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if constexpr (DT == MOE_F32)
                    w[j] = __float_as_uint(v[j]);
                else
                    w[j] = pack2<DT>(v[2 * j], v[2 * j + 1]);
            uint8_t *to = static_cast<uint8_t *>(x) + (row * stride + k) * (DT == MOE_F32 ? 4 : 2);
#pragma unroll
            for (int j = 0; j < 4; j += W / 4)
                if constexpr (W == 16)
                    *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
                else if constexpr (W == 8)
                    *reinterpret_cast<uint2 *>(to + 4 * j) = make_uint2(w[j], w[j + 1]);
                else
                    *reinterpret_cast<uint32_t *>(to + 4 * j) = w[j];
        } else {
#pragma unroll
            for (int j = 0; j < kEach; ++j)
                if (j < K - k)
                    store1<DT>(x, row * stride + k + j, v[j]);
        }
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
    uint32_t runs, units;   // of `run` elements in a row, and in all rows
    unsigned grid;
    int width, align;      // bytes that x's rows and the codes' rows are aligned to: 16, 8, 4 or 2; 4, 2 or 1
    Shape(const void *x, int64_t rows, int64_t K, int64_t stride, int size, const void *codes, int run)
    {
        runs = (uint32_t)((K + run - 1) / run);
        units = (uint32_t)rows * runs;   // check() has seen to it that they are below 2^31
        grid = (units + kThreads / 32 - 1) / (kThreads / 32);
        const uint64_t both = (uintptr_t)x | (uint64_t)(stride * size);
        width = both % 16 == 0 ? 16 : both % 8 == 0 ? 8 : both % 4 == 0 ? 4 : 2;
        const uint64_t either = (uintptr_t)codes | (uint64_t)(K / 2);
        align = either % 4 == 0 ? 4 : either % 2 == 0 ? 2 : 1;
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
    const Shape s(x, rows, K, stride, DT == MOE_F32 ? 4 : 2, codes, run_of<DT>());
    auto kernel = s.width == 16  ? quantize_any<DT, 16>
                  : s.width == 8 ? quantize_any<DT, 8>
                  : s.width == 4 || DT == MOE_F32 ? quantize_any<DT, 4> : quantize_any<DT, DT == MOE_F32 ? 4 : 2>;
    kernel<<<s.grid, kThreads, 0, st>>>(x, (int)K, stride, s.runs, s.units, s.align, codes, scales);
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
    const Shape s(x, rows, K, stride, DT == MOE_F32 ? 4 : 2, codes, run_of<DT>());
    auto kernel = s.width == 16  ? dequantize_any<DT, 16>
                  : s.width == 8 ? dequantize_any<DT, 8>
                  : s.width == 4 || DT == MOE_F32 ? dequantize_any<DT, 4> : dequantize_any<DT, DT == MOE_F32 ? 4 : 2>;
    kernel<<<s.grid, kThreads, 0, st>>>(codes, scales, (int)K, stride, s.runs, s.units, s.align, x);
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
