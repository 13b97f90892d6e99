// The experts' rows back to their tokens, weighted and summed, and the gradient of that
// (include/moe_tokens.h).
//
// Both read or write every row once and compute two operations an element, so HBM bounds them.  A token's row
// belongs to one group of threads, which goes through the columns with 64 or 128 bytes of loads a thread under way
// at once: of 8 rows, or of 4, 2 or 1 rows (where k is that small) in 2, 2 or 4 places.  The rows' places and their weights
// stay in registers (read again for each turn from L1: 378 against 331 us for 16384 x 7168 from 8 experts each).  Blocks are small and many and take tokens in order: what is read and written at a
// time then lies close together.
#include <string.h>

#include "rows.cuh"
#include "moe_tokens.h"
#include "ptx.cuh"

using namespace moe_mx;

namespace {

// most threads of a block (16384 x 7168 bfloat16, k = 8, each with its better launch bound: 32 threads 334 us, 64 317, 128 320, 256 342)
constexpr int kThreads = 64;
using moe_rows::kFull;

// W bytes of consecutive elements of DT, as they lie in memory
template <int DT, int W>
struct Piece {
    static constexpr int kElem = DT == MOE_F32 ? 4 : 2;
    static constexpr int kEach = W / kElem;
    static constexpr int kWords = (W + 3) / 4;
    uint32_t w[kWords];

    // (streamed: past L1)
    __device__ __forceinline__ void load(const void *base, int64_t i)
    {
        const uint8_t *p = static_cast<const uint8_t *>(base) + i * kElem;
        if constexpr (W == 16) {
            const uint4 q = mrr::ld_stream_v4(p);
            w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        } else if constexpr (W == 8) {
            asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[kWords - 1]) : "l"(p));
        } else if constexpr (W == 4) {
            asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
        } else {
            uint16_t h;
            asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(h) : "l"(p));
            w[0] = h;
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

__device__ __forceinline__ void store_weight(void *weight, int dt, int64_t i, float v)
{
    if (dt == MOE_F32)
        store1<MOE_F32>(weight, i, v);
    else if (dt == MOE_BF16)
        store1<MOE_BF16>(weight, i, v);
    else
        store1<MOE_F16>(weight, i, v);
}

struct Params {
    const void *rows, *weight, *grad_y;
    const int32_t *row_idx, *token_idx;
    void *y, *grad_rows, *grad_weight;
    int64_t T, R;
    int H, k, weight_dt;
    int group, tokens;   // threads of a token, tokens of a block
};

// pieces of W bytes that a thread has of each of R rows at once, `group` pieces apart (with pieces of 2 bytes, 32 in all:
// each takes a register)
template <int W, int R>
__host__ __device__ constexpr int pieces_at_once()
{
    return (R == 8 ? 1 : R == 1 ? 4 : 2) * (W >= 4 ? 16 / W : 4);
}

// Threads of a token whose row is `columns` threads' work: a power of two up to 16, else warps, at most `most`, and as
// few as take no more turns than those would.
int group_of(int64_t columns, int most)
{
    if (columns <= 16) {
        int g = 1;
        while (g < columns)
            g *= 2;
        return g;
    }
    const int64_t turns = (columns + most - 1) / most;
    return (int)(((columns + turns - 1) / turns + 31) / 32 * 32);
}

// slots j0 .. j0 + R - 1 of a token: their rows (-1: none) and weights
template <int R>
__device__ __forceinline__ void load_slots(const Params &p, int64_t t, int j0, int (&row)[R], float (&weight)[R])
{
#pragma unroll
    for (int j = 0; j < R; ++j) {
        row[j] = -1;
        weight[j] = 1.0f;
        if (j0 + j < p.k) {
            row[j] = __ldg(p.row_idx + t * p.k + j0 + j);
            row[j] = row[j] < p.R ? row[j] : -1;
            if (p.weight)
                weight[j] = load_weight(p.weight, p.weight_dt, t * p.k + j0 + j);
        }
    }
}

// y[t] where R slots at most, those in `mask`, have rows
template <int DT, int W, int R>
__device__ __forceinline__ void combine_few(const Params &p, int64_t t, int lane, uint32_t mask)
{
    using P = Piece<DT, W>;
    constexpr int U = pieces_at_once<W, R>();
    const int pieces = p.H / P::kEach;
    int row[R];
    float weight[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        row[j] = -1;
        weight[j] = 1.0f;
        if (mask) {
            const int64_t at = t * p.k + __ffs(mask) - 1;
            mask &= mask - 1;
            row[j] = __ldg(p.row_idx + at);
            if (p.weight)
                weight[j] = load_weight(p.weight, p.weight_dt, at);
        }
    }
    for (int c = blockIdx.y * U * p.group + lane; c < pieces; c += gridDim.y * U * p.group) {
        P v[R][U];
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (row[j] >= 0 && c + u * p.group < pieces)
                    v[j][u].load(p.rows, (int64_t)row[j] * p.H + (c + u * p.group) * P::kEach);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (c + u * p.group >= pieces)
                continue;
            float sum[P::kEach];
#pragma unroll
            for (int i = 0; i < P::kEach; ++i)
                sum[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (row[j] < 0)
                    continue;
                float f[P::kEach];
                v[j][u].get(f);
#pragma unroll
                for (int i = 0; i < P::kEach; ++i)
                    sum[i] = fmaf(weight[j], f[i], sum[i]);
            }
            P out;
            out.set(sum);
            out.store(p.y, t * p.H + (c + u * p.group) * P::kEach);
        }
    }
}

// R rows at once.  Where tokens are few, several blocks (the y index) share a token's columns.
// (Of 8 rows in pieces of 16 bytes 11 blocks an SM: for 12 a register is spilled, 319 us for 317 at 16384 x 7168.)
template <int DT, int W, int R>
__global__ void __launch_bounds__(kThreads, W == 16 && R == 8 ? 11 : W > 2 ? 12 : 8) combine(Params p)
{
    using P = Piece<DT, W>;
    constexpr int U = pieces_at_once<W, R>();
    const int of_block = threadIdx.x / p.group, lane = threadIdx.x - of_block * p.group;
    const int64_t t = (int64_t)blockIdx.x * p.tokens + of_block;
    if (t >= p.T)
        return;
    // A token that has rows in few of its slots (its other experts are held elsewhere) has more of each row under way (16384 x
    // 7168, 8 experts each, a quarter of them held: 121 us, 159 without; an eighth: 87 and 134; 8192 x 2049 float16, a quarter:
    // 46 and 75).  Pieces of 4 bytes stay as they are: with all forms in one kernel 8192 x 2050 with every row takes
    // 72 us instead of 64.
    if (W != 4 && R > 1 && p.k <= R && p.group >= 32) {
        uint32_t mask = 0u;
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (j < p.k) {
                const int at = __ldg(p.row_idx + t * p.k + j);
                mask |= at >= 0 && at < p.R ? 1u << j : 0u;
            }
        const int n = __popc(mask);
        if (n <= 1)
            return combine_few<DT, W, 1>(p, t, lane, mask);
        if (R > 2 && n <= 2)
            return combine_few<DT, W, 2>(p, t, lane, mask);
        if (R > 4 && n <= 4)
            return combine_few<DT, W, 4>(p, t, lane, mask);
    }
    const int pieces = p.H / P::kEach;
    int row[R];
    float weight[R];
    load_slots<R>(p, t, 0, row, weight);
    for (int c = blockIdx.y * U * p.group + lane; c < pieces; c += gridDim.y * U * p.group) {
        float sum[U][P::kEach];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < P::kEach; ++i)
                sum[u][i] = 0.0f;
        for (int j0 = 0; j0 < p.k; j0 += R) {
            if (p.k > R)
                load_slots<R>(p, t, j0, row, weight);
            P v[R][U];
#pragma unroll
            for (int j = 0; j < R; ++j)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (row[j] >= 0 && c + u * p.group < pieces)
                        v[j][u].load(p.rows, (int64_t)row[j] * p.H + (c + u * p.group) * P::kEach);
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (row[j] < 0)
                    continue;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float f[P::kEach];
                    v[j][u].get(f);
#pragma unroll
                    for (int i = 0; i < P::kEach; ++i)
                        sum[u][i] = fmaf(weight[j], f[i], sum[u][i]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * p.group < pieces) {
                P out;
                out.set(sum[u]);
                out.store(p.y, t * p.H + (c + u * p.group) * P::kEach);
            }
    }
}

// A thread's sums of R slots stay while it goes through the columns.  The blocks behind the tokens' write the rows of
// zeros, each every `zero_blocks`th row: these rows follow one another.  Few rows go to as many warps as there are.
template <int DT, int W, int R, int THREADS>
__global__ void __launch_bounds__(THREADS, (W == 16 ? 640 : 512) / THREADS) combine_grad(Params p)
{
    using P = Piece<DT, W>;
    constexpr int U = pieces_at_once<W, R>();
    __shared__ float part[THREADS / 32][R];
    const int lane32 = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int pieces = p.H / P::kEach;
    const int64_t token_blocks = (p.T + p.tokens - 1) / p.tokens;
    if (blockIdx.x >= token_blocks) {
        const int64_t zero_blocks = gridDim.x - token_blocks;
        const bool few = zero_blocks * blockDim.x >= 2 * p.R;
        const int64_t mine = blockIdx.x - token_blocks + (few ? lane32 * (blockDim.x / 32) + warp : threadIdx.x) * zero_blocks;
        uint32_t none = __ballot_sync(kFull, mine < p.R && __ldg(p.token_idx + min(mine, p.R - 1)) < 0);
        while (none) {
            const int64_t r = __shfl_sync(kFull, mine, __ffs(none) - 1);
            none &= none - 1;
            moe_rows::clear<P::kElem>(p.grad_rows, r * p.H, p.H, lane32, 32);
        }
        return;
    }
    const int of_block = threadIdx.x / p.group, lane = threadIdx.x - of_block * p.group;
    const int64_t t = (int64_t)blockIdx.x * p.tokens + of_block;
    const bool mine = t < p.T;   // the whole block stays for its barriers
    for (int j0 = 0; j0 < p.k; j0 += R) {
        int row[R];
        float weight[R], sum[R];
#pragma unroll
        for (int j = 0; j < R; ++j)
            sum[j] = 0.0f;
        if (mine)
            load_slots<R>(p, t, j0, row, weight);
        for (int c = lane; mine && c < pieces; c += U * p.group) {
            P g[U], v[R][U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c + u * p.group < pieces)
                    g[u].load(p.grad_y, t * p.H + (c + u * p.group) * P::kEach);
            if (p.grad_weight) {
#pragma unroll
                for (int j = 0; j < R; ++j)
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (row[j] >= 0 && c + u * p.group < pieces)
                            v[j][u].load(p.rows, (int64_t)row[j] * p.H + (c + u * p.group) * P::kEach);
            }
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (row[j] < 0)
                    continue;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (c + u * p.group >= pieces)
                        continue;
                    float f[P::kEach], x[P::kEach];
                    g[u].get(f);
                    if (p.grad_weight) {
                        v[j][u].get(x);
#pragma unroll
                        for (int i = 0; i < P::kEach; ++i)
                            sum[j] = fmaf(f[i], x[i], sum[j]);
                    }
#pragma unroll
                    for (int i = 0; i < P::kEach; ++i)
                        x[i] = weight[j] * f[i];
                    P out;
                    out.set(x);
                    out.store(p.grad_rows, (int64_t)row[j] * p.H + (c + u * p.group) * P::kEach);
                }
            }
        }
        if (!p.grad_weight)
            continue;
        // over the token's threads: inside a warp by shuffles, warps through shared memory
        const int width = min(p.group, 32);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            for (int d = width / 2; d > 0; d /= 2)
                sum[j] += __shfl_xor_sync(kFull, sum[j], d);
            if (p.group >= 32 && lane32 == 0)
                part[warp][j] = sum[j];
        }
        __syncthreads();
        if (mine && lane < R && p.group >= 32 && j0 + lane < p.k) {
            float s = 0.0f;
            for (int w = 0; w < p.group / 32; ++w)
                s += part[warp + w][lane];
            store_weight(p.grad_weight, p.weight_dt, t * p.k + j0 + lane, s);
        } else if (mine && p.group < 32 && lane == 0) {
#pragma unroll
            for (int j = 0; j < R; ++j)
                if (j0 + j < p.k)
                    store_weight(p.grad_weight, p.weight_dt, t * p.k + j0 + j, sum[j]);
        }
        __syncthreads();
    }
}

constexpr int kFewTokens = 304;        // for the gradient
constexpr int kZeroBlocks = 16 * 152;
constexpr int kFewBlocks = 4 * 152;    // fewer than these of one group each leave SMs idle

template <int DT, int W, int R, int THREADS>
void launch_grad(Params p, cudaStream_t st)
{
    const int64_t columns = p.H / Piece<DT, W>::kEach, at_once = pieces_at_once<W, R>();
    p.group = group_of((columns + at_once - 1) / at_once, THREADS);
    p.tokens = THREADS / p.group;
    const int threads = p.group * p.tokens;   // whole warps
    // behind the tokens' blocks, one for each `threads` rows (32 or more); few rows are spread over more (64 x 7168, 8
    // experts each, an eighth of them held: 7.7 us, 35 without; 4095 x 7168: 112 and 137)
    int64_t zero_blocks = (p.R + threads - 1) / threads;
    if (zero_blocks < kZeroBlocks)
        zero_blocks = p.R < kZeroBlocks ? p.R : kZeroBlocks;
    const int64_t blocks = (p.T + p.tokens - 1) / p.tokens + zero_blocks;
    combine_grad<DT, W, R, THREADS><<<(unsigned)blocks, threads, 0, st>>>(p);
}

template <int DT, int W, int R>
void launch(Params p, bool grad, cudaStream_t st)
{
    if (grad) {
        // few tokens: more threads to each (1 token of 7168 from 8 experts: 8.6 us with 256 threads, 16.5 with 64; 64
        // tokens 10.5 and 20.5; 400 tokens 22.8 and 24.8; 500 of 2048 from 2 experts 10.2 and 6.5)
        if (R == 8 && p.T < kFewTokens)
            launch_grad<DT, W, R, R == 8 ? 256 : kThreads>(p, st);
        else
            launch_grad<DT, W, R, kThreads>(p, st);
        return;
    }
    const int64_t pieces = p.H / Piece<DT, W>::kEach, at_once = pieces_at_once<W, R>(), columns = (pieces + at_once - 1) / at_once;
    p.group = group_of(columns, kThreads);
    p.tokens = kThreads / p.group;
    const int64_t blocks = (p.T + p.tokens - 1) / p.tokens;
    if (blocks == 0)
        return;
    // (3 tokens of 5120: 4.8 us, and 11.2 without sharing a row; 64 of 7168: 6.8 and 14.3)
    const int64_t turns = (columns + p.group - 1) / p.group, want = blocks < kFewBlocks ? kFewBlocks / blocks : 1;
    combine<DT, W, R><<<dim3((unsigned)blocks, (unsigned)(turns < want ? turns : want)), p.group * p.tokens, 0, st>>>(p);
}

template <int DT, int W>
void launch(const Params &p, bool grad, cudaStream_t st)
{
    if (p.k > 4 || (grad && p.T < kFewTokens))
        launch<DT, W, 8>(p, grad, st);
    else if (p.k > 2)
        launch<DT, W, 4>(p, grad, st);
    else if (p.k > 1)
        launch<DT, W, 2>(p, grad, st);
    else
        launch<DT, W, 1>(p, grad, st);
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
    // at most 2^31 - 1 blocks: one or more tokens each, and behind them kZeroBlocks or blocks for 32 or more rows each
    const bool ok = T >= 0 && R >= 0 && T <= INT32_MAX && R <= INT32_MAX && H >= 1 && H <= (1 << 20) && k >= 1 &&
                    k <= MOE_SORT_MAX_K && T + R / 32 < INT32_MAX - kZeroBlocks;
    return ok ? MRR_OK : MRR_ERR_SHAPE;
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
