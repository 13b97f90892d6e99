// The experts' rows back to their tokens, weighted and summed, and the gradient of that
// (include/moe_tokens.h).
//
// Both read or write every row once and compute two operations an element, so HBM bounds them.
#include <string.h>

#include "mx.cuh"
#include "moe_tokens.h"

using namespace moe_mx;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kRows = 8;   // rows of a token loaded before the first is used

// W bytes of consecutive elements of DT, as they lie in memory
template <int DT, int W>
struct Piece {
    static constexpr int kElem = DT == MOE_F32 ? 4 : 2;
    static constexpr int kEach = W / kElem;
    static constexpr int kWords = (W + 3) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const void *base, int64_t i)
    {
        const uint8_t *p = static_cast<const uint8_t *>(base) + i * kElem;
        if constexpr (W == 16) {
            const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p));
            w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        } else if constexpr (W == 8) {
            const uint2 q = __ldg(reinterpret_cast<const uint2 *>(p));
            w[0] = q.x, w[1] = q.y;
        } else if constexpr (W == 4) {
            w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
        } else {
            w[0] = __ldg(reinterpret_cast<const uint16_t *>(p));
        }
    }

    __device__ __forceinline__ void store(void *base, int64_t i) const
    {
        uint8_t *p = static_cast<uint8_t *>(base) + i * kElem;
        if constexpr (W == 16)
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (W == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else if constexpr (W == 4)
            *reinterpret_cast<uint32_t *>(p) = w[0];
        else
            *reinterpret_cast<uint16_t *>(p) = (uint16_t)w[0];
    }

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            w[i] = 0u;
    }

    __device__ __forceinline__ void get(float (&v)[kEach]) const
    {
        if constexpr (DT == MOE_F32) {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const float2 f = unpack2<DT>(w[i]);
                v[2 * i] = f.x;
                if constexpr (kEach > 1)
                    v[2 * i + 1] = f.y;
            }
        }
    }

    __device__ __forceinline__ void set(const float (&v)[kEach])
    {
        if constexpr (DT == MOE_F32) {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = pack2<DT>(v[2 * i], kEach > 1 ? v[kEach > 1 ? 2 * i + 1 : 0] : 0.0f);
        }
    }
};

__device__ __forceinline__ float load_weight(const void *weight, int dt, int64_t i)
{
    return dt == MOE_F32 ? load1<MOE_F32>(weight, i) : dt == MOE_BF16 ? load1<MOE_BF16>(weight, i) : load1<MOE_F16>(weight, i);
}

struct Params {
    const void *rows, *weight, *grad_y;
    const int32_t *row_idx, *token_idx;
    void *y, *grad_rows, *grad_weight;
    int64_t T, R;
    int H, k, weight_dt, segs;
};

// A warp has 32 pieces of one token.  The token's rows and weights are loaded by the lanes, one each, and
// passed round; the rows' pieces are loaded kRows at a time.
template <int DT, int W>
__global__ void __launch_bounds__(kThreads) combine(Params p)
{
    using P = Piece<DT, W>;
    const int lane = threadIdx.x % 32;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    const int64_t t = unit / p.segs;
    if (t >= p.T)
        return;
    const int c = ((int)(unit - t * p.segs) * 32 + lane) * P::kEach;
    const bool mine = c < p.H;
    float sum[P::kEach];
#pragma unroll
    for (int i = 0; i < P::kEach; ++i)
        sum[i] = 0.0f;
    for (int j0 = 0; j0 < p.k; j0 += 32) {
        int64_t row = -1;
        float weight = 1.0f;
        if (j0 + lane < p.k) {
            row = __ldg(p.row_idx + t * p.k + j0 + lane);
            row = row < p.R ? row : -1;
            if (p.weight)
                weight = load_weight(p.weight, p.weight_dt, t * p.k + j0 + lane);
        }
        const int count = min(32, p.k - j0);
        for (int j1 = 0; j1 < count; j1 += kRows) {
            P v[kRows];
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                const int r = __shfl_sync(kFull, (int)row, min(j1 + j, 31));
                if (j1 + j < count && r >= 0 && mine)
                    v[j].load(p.rows, (int64_t)r * p.H + c);
            }
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                const int r = __shfl_sync(kFull, (int)row, min(j1 + j, 31));
                const float w = __shfl_sync(kFull, weight, min(j1 + j, 31));
                if (j1 + j < count && r >= 0 && mine) {
                    float f[P::kEach];
                    v[j].get(f);
#pragma unroll
                    for (int i = 0; i < P::kEach; ++i)
                        sum[i] = fmaf(w, f[i], sum[i]);
                }
            }
        }
    }
    if (mine) {
        P out;
        out.set(sum);
        out.store(p.y, t * p.H + c);
    }
}

// One block for each token, and behind them blocks that write the rows of zeros.  Each thread holds its pieces of
// grad_y while it goes through kSlots of the token's rows, and one of the sums of each.
constexpr int kSlots = 8;

template <int DT, int W>
__global__ void __launch_bounds__(kThreads) combine_grad(Params p)
{
    using P = Piece<DT, W>;
    __shared__ float part[kWarps][kSlots];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int pieces = p.H / P::kEach;
    if (blockIdx.x >= p.T) {
        const int64_t r0 = ((int64_t)blockIdx.x - p.T) * kThreads + threadIdx.x;
        uint32_t none = __ballot_sync(kFull, r0 < p.R && __ldg(p.token_idx + min(r0, p.R - 1)) < 0);
        while (none) {
            const int64_t r = r0 - lane + __ffs(none) - 1;
            none &= none - 1;
            P z;
            z.zero();
            for (int c = lane; c < pieces; c += 32)
                z.store(p.grad_rows, r * p.H + (int64_t)c * P::kEach);
        }
        return;
    }
    const int64_t t = blockIdx.x;
    for (int j0 = 0; j0 < p.k; j0 += kSlots) {
        int64_t row[kSlots];
        float weight[kSlots], sum[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            row[j] = -1;
            weight[j] = 1.0f;
            sum[j] = 0.0f;
            if (j0 + j < p.k) {
                row[j] = __ldg(p.row_idx + t * p.k + j0 + j);
                row[j] = row[j] < p.R ? row[j] : -1;
                if (p.weight)
                    weight[j] = load_weight(p.weight, p.weight_dt, t * p.k + j0 + j);
            }
        }
        for (int c = threadIdx.x; c < pieces; c += kThreads) {
            P g, v[kSlots];
            g.load(p.grad_y, t * p.H + (int64_t)c * P::kEach);
            if (p.grad_weight) {
#pragma unroll
                for (int j = 0; j < kSlots; ++j)
                    if (row[j] >= 0)
                        v[j].load(p.rows, row[j] * p.H + (int64_t)c * P::kEach);
            }
            float f[P::kEach];
            g.get(f);
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                if (row[j] < 0)
                    continue;
                float x[P::kEach];
                if (p.grad_weight) {
                    v[j].get(x);
#pragma unroll
                    for (int i = 0; i < P::kEach; ++i)
                        sum[j] = fmaf(f[i], x[i], sum[j]);
                }
#pragma unroll
                for (int i = 0; i < P::kEach; ++i)
                    x[i] = weight[j] * f[i];
                P out;
                out.set(x);
                out.store(p.grad_rows, row[j] * p.H + (int64_t)c * P::kEach);
            }
        }
        if (!p.grad_weight)
            continue;
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            float s = sum[j];
#pragma unroll
            for (int d = 16; d > 0; d /= 2)
                s += __shfl_xor_sync(kFull, s, d);
            if (lane == 0)
                part[warp][j] = s;
        }
        __syncthreads();
        if (threadIdx.x < kSlots && j0 + (int)threadIdx.x < p.k) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                s += part[w][threadIdx.x];
            const int64_t at = t * p.k + j0 + threadIdx.x;
            if (p.weight_dt == MOE_F32)
                store1<MOE_F32>(p.grad_weight, at, s);
            else if (p.weight_dt == MOE_BF16)
                store1<MOE_BF16>(p.grad_weight, at, s);
            else
                store1<MOE_F16>(p.grad_weight, at, s);
        }
        __syncthreads();
    }
}

template <int DT, int W>
void launch(Params p, bool grad, cudaStream_t st)
{
    if (grad) {
        const int64_t blocks = p.T + (p.token_idx ? (p.R + kThreads - 1) / kThreads : 0);
        combine_grad<DT, W><<<(unsigned)blocks, kThreads, 0, st>>>(p);
        return;
    }
    constexpr int kEach = Piece<DT, W>::kEach;
    p.segs = (p.H + 32 * kEach - 1) / (32 * kEach);
    const int64_t units = p.T * p.segs;
    combine<DT, W><<<(unsigned)((units + kWarps - 1) / kWarps), kThreads, 0, st>>>(p);
}

template <int DT>
void launch(const Params &p, uintptr_t all, bool grad, cudaStream_t st)
{
    if (all % 16 == 0)
        launch<DT, 16>(p, grad, st);
    else if (all % 8 == 0)
        launch<DT, 8>(p, grad, st);
    else if (all % 4 == 0 || DT == MOE_F32)
        launch<DT, 4>(p, grad, st);
    else
        launch<DT, DT == MOE_F32 ? 4 : 2>(p, grad, st);
}

bool aligned(const void *p, uintptr_t n) { return (uintptr_t)p % n == 0; }
bool is_float(moe_dtype dt) { return dt == MOE_F16 || dt == MOE_BF16 || dt == MOE_F32; }
uintptr_t size_of(moe_dtype dt) { return dt == MOE_F32 ? 4 : 2; }

mrr_status run(Params &p, moe_dtype dt, uintptr_t pointers, bool grad, mrr_stream_t stream)
{
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const uintptr_t all = pointers | (uintptr_t)p.H * size_of(dt);
    if (dt == MOE_F32)
        launch<MOE_F32>(p, all, grad, st);
    else if (dt == MOE_BF16)
        launch<MOE_BF16>(p, all, grad, st);
    else
        launch<MOE_F16>(p, all, grad, st);
    return cudaGetLastError() == cudaSuccess ? MRR_OK : MRR_ERR_CUDA;
}

mrr_status check(moe_dtype dt, int64_t R, int64_t H, int64_t T, int64_t k, const void *weight, moe_dtype weight_dt)
{
    if (!is_float(dt) || (weight && !is_float(weight_dt)))
        return MRR_ERR_DTYPE;
    // at most 2^31 - 1 blocks: a warp has a piece of 64 elements or more, or a block a token
    if (T < 0 || R < 0 || T > INT32_MAX || R > INT32_MAX || H < 1 || H > (1 << 20) || k < 1 ||
        k > MOE_SORT_MAX_K || (T + 1) * ((H + 31) / 32) > 8ll * INT32_MAX || T + R / kThreads + 1 > INT32_MAX)
        return MRR_ERR_SHAPE;
    return MRR_OK;
}

}  // namespace

extern "C" {

mrr_status moe_combine_run(const void *rows, moe_dtype dt, int64_t R, int64_t H, const int32_t *row_idx, int64_t T,
                           int64_t k, const void *weight, moe_dtype weight_dt, void *y, mrr_stream_t stream)
{
    const mrr_status bad = check(dt, R, H, T, k, weight, weight_dt);
    if (bad != MRR_OK)
        return bad;
    if (T > 0 && (!row_idx || !y || (R > 0 && !rows)))
        return MRR_ERR_NULL;
    if (!aligned(rows, size_of(dt)) || !aligned(y, size_of(dt)) || !aligned(row_idx, 4) ||
        (weight && !aligned(weight, size_of(weight_dt))))
        return MRR_ERR_ALIGN;
    if (T == 0)
        return MRR_OK;
    Params p;
    memset(&p, 0, sizeof(p));
    p.rows = rows;
    p.weight = weight;
    p.weight_dt = weight_dt;
    p.row_idx = row_idx;
    p.y = y;
    p.T = T;
    p.R = R;
    p.H = (int)H;
    p.k = (int)k;
    return run(p, dt, (uintptr_t)rows | (uintptr_t)y, false, stream);
}

mrr_status moe_combine_grad_run(const void *grad_y, const void *rows, moe_dtype dt, int64_t R, int64_t H,
                                const int32_t *row_idx, const int32_t *token_idx, int64_t T, int64_t k,
                                const void *weight, moe_dtype weight_dt, void *grad_rows, void *grad_weight,
                                mrr_stream_t stream)
{
    const mrr_status bad = check(dt, R, H, T, k, weight, weight_dt);
    if (bad != MRR_OK)
        return bad;
    if ((T > 0 && (!grad_y || !row_idx)) || (R > 0 && (!token_idx || !grad_rows)) ||
        (grad_weight && (!weight || (R > 0 && !rows))))
        return MRR_ERR_NULL;
    if (!aligned(rows, size_of(dt)) || !aligned(grad_y, size_of(dt)) || !aligned(grad_rows, size_of(dt)) ||
        !aligned(row_idx, 4) || !aligned(token_idx, 4) || (weight && !aligned(weight, size_of(weight_dt))) ||
        (grad_weight && !aligned(grad_weight, size_of(weight_dt))))
        return MRR_ERR_ALIGN;
    if (T == 0 && R == 0)
        return MRR_OK;
    Params p;
    memset(&p, 0, sizeof(p));
    p.rows = grad_weight ? rows : nullptr;
    p.grad_y = grad_y;
    p.weight = weight;
    p.weight_dt = weight_dt;
    p.row_idx = row_idx;
    p.token_idx = token_idx;
    p.grad_rows = grad_rows;
    p.grad_weight = grad_weight;
    p.T = T;
    p.R = R;
    p.H = (int)H;
    p.k = (int)k;
    return run(p, dt, (uintptr_t)p.rows | (uintptr_t)grad_y | (uintptr_t)grad_rows, true, stream);
}

}  // extern "C"
