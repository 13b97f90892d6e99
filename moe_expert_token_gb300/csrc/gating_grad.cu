// The gradient of the MoE gating top-k op (include/moe_gating_grad.h).
//
// The gradient of the scores has k numbers of a token's own, at the chosen experts, beside grad_norm_out's, which is dense.
// A group of lanes has a token, a lane a chosen expert (two where k is above 32), whose logit it reads where it lies.
//   * Scores that stand alone (sigmoid, softplus) without grad_norm_out: the rest of grad_x is zero.  Several tokens
//     share a warp, which writes their rows of zeros ahead of the k values.
//   * Else (N > 0) a warp has a token and its row of logits in registers: softmax needs its sum, and every element gets
//     score * (grad_norm_out - dot) or the like; the k values are written over it afterwards.
// Each element is read or written once with an exponential between: for the usual sizes (16384 rows of 256 in 16 bits, 8 to
// 17 MB) launches and the latency of a row count for as much as HBM.  16384 x 256 bfloat16: sigmoid 4.6 us, with a bias 7.5; softmax
// 11.4 and 17.8, where the instructions of a row's sums count most: two slots a lane, of which a token of 8 experts uses a quarter
// of one, and shuffles that wait for each other.
//
// The gradient of the biases is a sum over rows: warps hold sums of their own in shared memory while the block goes from
// row to row, each block leaves one row of partial sums, and a second launch adds those in order.
#include <atomic>
#include <string.h>

#include "column_sum.cuh"
#include "device_info.h"
#include "moe_gating_grad.h"

using namespace moe_rows;

static_assert((int)MRR_GATE_F16 == (int)MOE_F16 && (int)MRR_GATE_BF16 == (int)MOE_BF16 && (int)MRR_GATE_F32 == (int)MOE_F32,
              "one set of type codes");

namespace {

constexpr int kWarps = 8;
constexpr int kMaxBlocks = 304;   // two on each of the 152 SMs

struct Params {
    const void *grad_y, *x, *bias, *extra_bias;
    const int32_t *expert_idx;
    const uint8_t *extra_mask;
    const float *grad_norm;
    void *grad_x;
    float *partial;    // [blocks][2][e], or NULL
    int64_t T;
    int e, k, norm_type;
    float scale, eps;
};

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// d score / d x of a score that stands alone: s (1 - s), without the cancellation of 1 - s, or the sigmoid
__device__ __forceinline__ float slope_of(int norm_type, float x)
{
    if (norm_type == 2)
        return sigmoid(x);
    const float z = expf(-fabsf(x)), n = 1.0f + z;
    return z / (n * n);
}

// softmax is x's exponential over the row's sum (top: the row's largest); softplus log(1 + exp(x))
__device__ __forceinline__ float score_of(int norm_type, float x, float top, float sum)
{
    if (norm_type == 0)
        return expf(x - top) / sum;
    if (norm_type == 1)
        return sigmoid(x);
    return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x)));
}

// V consecutive elements of a row, from an address aligned to them
template <int DT, int V>
__device__ __forceinline__ void load_group(const void *base, int64_t i, float (&v)[V])
{
    if constexpr (V == 1) {
        v[0] = load1<DT>(base, i);
    } else if constexpr (DT == MOE_F32) {
        const float4 q = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(base) + i));
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else {
        const uint2 q = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + i));
        const float2 lo = unpack2<DT>(q.x), hi = unpack2<DT>(q.y);
        v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
    }
}

template <int DT, int V>
__device__ __forceinline__ void store_group(void *base, int64_t i, const float (&v)[V])
{
    if constexpr (V == 1)
        store1<DT>(base, i, v[0]);
    else if constexpr (DT == MOE_F32)
        *reinterpret_cast<float4 *>(static_cast<float *>(base) + i) = make_float4(v[0], v[1], v[2], v[3]);
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(base) + i) = make_uint2(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]));
}

// LANES lanes a token (k <= LANES; 32 lanes: two slots each).  N > 0 (with 32 lanes): N groups of V elements of the row a
// lane.  Shared memory: [1 or 2][e] sums of each warp, where bias gradients are asked for.
template <int DT, int LANES, int N, int V>
__global__ void __launch_bounds__(32 * kWarps) gating_grad(Params p)
{
    extern __shared__ float sums[];
    mrr::grid_launch_dependents();
    constexpr int kSlots = LANES == 32 ? 2 : 1, kTokens = 32 / LANES;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, of_warp = lane / LANES, at = lane % LANES;
    const int kinds = p.extra_mask ? 2 : 1;
    float *mine = sums + warp * kinds * p.e;
    if (p.partial) {
        for (int i = lane; i < kinds * p.e; i += 32)
            mine[i] = 0.0f;
        __syncwarp();
    }
    for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * kTokens; t0 < p.T; t0 += (int64_t)gridDim.x * kWarps * kTokens) {
        const int64_t t = t0 + of_warp;
        const bool here = t < p.T;
        const bool extra = here && p.extra_mask && p.extra_mask[t] != 0;
        const void *bias = extra ? p.extra_bias : p.bias;
        int idx[kSlots];
        float g[kSlots], x[kSlots], n[kSlots], d[kSlots], sum = 0.0f, inner = 0.0f;
#pragma unroll
        for (int h = 0; h < kSlots; ++h) {
            const int j = LANES * h + at;
            const bool in = here && j < p.k;
            idx[h] = in ? __ldg(p.expert_idx + t * p.k + j) : -1;
            g[h] = in ? load1<DT>(p.grad_y, t * p.k + j) : 0.0f;
            if (idx[h] < 0 || idx[h] >= p.e)
                idx[h] = -1, g[h] = 0.0f;
        }
#pragma unroll
        for (int h = 0; h < kSlots; ++h)
            x[h] = idx[h] >= 0 ? load1<DT>(p.x, t * p.e + idx[h]) : 0.0f;
        // the row: its scores, for softmax without their common factor
        float row[N > 0 ? N : 1][V];
        float top = 0.0f, total = 1.0f;
        if constexpr (N > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (32 * i + lane) * V;
                if (c < p.e)
                    load_group<DT, V>(p.x, t * p.e + c, row[i]);
            }
            if (p.norm_type == 0) {
                top = -INFINITY;
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int u = 0; u < V; ++u)
                        top = (32 * i + lane) * V < p.e ? fmaxf(top, row[i][u]) : top;
#pragma unroll
                for (int o = 16; o > 0; o /= 2)
                    top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
                total = 0.0f;
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int u = 0; u < V; ++u) {
                        row[i][u] = (32 * i + lane) * V < p.e ? expf(row[i][u] - top) : 0.0f;
                        total += row[i][u];
                    }
                total = warp_sum(total);
            }
        } else {
            clear<DT == MOE_F32 ? 4 : 2>(p.grad_x, t0 * p.e, min((int64_t)kTokens, p.T - t0) * p.e, lane, 32);
        }
#pragma unroll
        for (int h = 0; h < kSlots; ++h) {
            n[h] = idx[h] >= 0 ? score_of(p.norm_type, x[h], top, total) : 0.0f;
            const float s = n[h] + (bias && idx[h] >= 0 ? load1<DT>(bias, idx[h]) : 0.0f);
            sum += s;
            inner = fmaf(g[h], s, inner);
        }
#pragma unroll
        for (int o = LANES / 2; o > 0; o /= 2) {
            sum += __shfl_xor_sync(kFull, sum, o);
            inner += __shfl_xor_sync(kFull, inner, o);
        }
        sum += p.eps;
        const float factor = p.scale / sum;
        inner /= sum;
#pragma unroll
        for (int h = 0; h < kSlots; ++h)
            d[h] = idx[h] >= 0 ? factor * (g[h] - inner) : 0.0f;
        // an expert that a token has twice (hash routing): its first slot gets the sum, in the order of the slots
        bool twice = false;
#pragma unroll
        for (int h = 0; h < kSlots; ++h) {
            const uint32_t group = LANES == 32 ? kFull : ((1u << LANES) - 1) << (of_warp * LANES);
            const uint32_t same = __match_any_sync(kFull, idx[h]) & group;
            twice |= idx[h] >= 0 && __popc(same) > 1;
        }
        if (__any_sync(kFull, twice || p.k > 32)) {   // (slots 32 and above are not compared with the others here)
            float all[kSlots];
            bool first[kSlots];
#pragma unroll
            for (int h = 0; h < kSlots; ++h)
                all[h] = 0.0f, first[h] = true;
#pragma unroll
            for (int o = 0; o < kSlots; ++o)
#pragma unroll 1
                for (int l = 0; l < LANES; ++l) {
                    const int other = __shfl_sync(kFull, idx[o], of_warp * LANES + l);
                    const float share = __shfl_sync(kFull, d[o], of_warp * LANES + l);
#pragma unroll
                    for (int h = 0; h < kSlots; ++h)
                        if (other == idx[h]) {
                            all[h] += share;
                            if (LANES * o + l < LANES * h + at)
                                first[h] = false;
                        }
                }
#pragma unroll
            for (int h = 0; h < kSlots; ++h) {
                d[h] = all[h];
                if (!first[h])
                    idx[h] = -1, d[h] = 0.0f;
            }
        }
        float dot = 0.0f;
        if constexpr (N > 0) {
            const float *norm = p.grad_norm + t * p.e;   // (not read where there is none)
            const float per = 1.0f / total;
            float more[V];
            if (p.norm_type == 0) {
#pragma unroll
                for (int h = 0; h < kSlots; ++h)
                    dot = fmaf(d[h], n[h], dot);
                if (p.grad_norm) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int c = (32 * i + lane) * V;
                        if (c < p.e) {
                            load_group<MOE_F32, V>(norm, c, more);
#pragma unroll
                            for (int u = 0; u < V; ++u)
                                dot = fmaf(more[u], row[i][u] * per, dot);
                        }
                    }
                }
                dot = warp_sum(dot);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = (32 * i + lane) * V;
                if (c >= p.e)
                    continue;
#pragma unroll
                for (int u = 0; u < V; ++u)
                    more[u] = 0.0f;
                if (p.grad_norm)
                    load_group<MOE_F32, V>(norm, c, more);
                float out[V];
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    out[u] = p.norm_type == 0 ? row[i][u] * per * (more[u] - dot) : more[u] * slope_of(p.norm_type, row[i][u]);
                    if (p.partial && p.grad_norm)
                        mine[(extra ? p.e : 0) + c + u] += more[u];
                }
                store_group<DT, V>(p.grad_x, t * p.e + c, out);
            }
        }
        __syncwarp();   // the rest of the rows is written
#pragma unroll
        for (int h = 0; h < kSlots; ++h)
            if (idx[h] >= 0) {
                const float ds = d[h] + (N > 0 && p.grad_norm ? __ldg(p.grad_norm + t * p.e + idx[h]) : 0.0f);
                const float out = p.norm_type == 0 ? n[h] * (ds - dot) : ds * slope_of(p.norm_type, x[h]);
                store1<DT>(p.grad_x, t * p.e + idx[h], out);
            }
        if (p.partial) {
            // one token after the other: two of them may have the same expert
#pragma unroll
            for (int w = 0; w < kTokens; ++w) {
                if (w == of_warp) {
#pragma unroll
                    for (int h = 0; h < kSlots; ++h)
                        if (idx[h] >= 0)
                            mine[(extra ? p.e : 0) + idx[h]] += d[h];
                }
                __syncwarp();
            }
        }
    }
    if (!p.partial)
        return;
    __syncthreads();
    for (int i = threadIdx.x; i < kinds * p.e; i += 32 * kWarps) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            s += sums[w * kinds * p.e + i];
        p.partial[(int64_t)blockIdx.x * 2 * p.e + i] = s;
    }
}

// with bias gradients the blocks stay for many rows, else there are as many as rows ask for
int64_t blocks_for(int64_t T)
{
    const int64_t blocks = (T + kWarps - 1) / kWarps;
    return blocks < kMaxBlocks ? blocks : kMaxBlocks;
}

template <int DT, int LANES, int N, int V>
cudaError_t launch(const Params &p, cudaStream_t st)
{
    static std::atomic<uint64_t> done;
    mrr_device::Info info;
    if (!mrr_device::current(info))
        return cudaErrorUnknown;
    const int smem = p.partial ? kWarps * (p.extra_mask ? 2 : 1) * p.e * 4 : 0;   // up to 64 KB
    const cudaError_t err = mrr_device::allow_smem(gating_grad<DT, LANES, N, V>, info, done);
    if (err != cudaSuccess)
        return err;
    const int64_t rows = kWarps * (32 / LANES), blocks = p.partial ? blocks_for(p.T) : (p.T + rows - 1) / rows;
    gating_grad<DT, LANES, N, V><<<(unsigned)blocks, 32 * kWarps, smem, st>>>(p);
    return cudaGetLastError();
}

template <int DT>
cudaError_t launch(const Params &p, bool wide, cudaStream_t st)
{
    if (p.norm_type != 0 && !p.grad_norm)
        return p.k <= 8    ? launch<DT, 8, 0, 1>(p, st)
               : p.k <= 16 ? launch<DT, 16, 0, 1>(p, st)
                           : launch<DT, 32, 0, 1>(p, st);
    if (wide)
        return p.e <= 128   ? launch<DT, 32, 1, 4>(p, st)
               : p.e <= 256 ? launch<DT, 32, 2, 4>(p, st)
               : p.e <= 512 ? launch<DT, 32, 4, 4>(p, st)
                            : launch<DT, 32, 8, 4>(p, st);
    return p.e <= 128 ? launch<DT, 32, 4, 1>(p, st) : p.e <= 512 ? launch<DT, 32, 16, 1>(p, st) : launch<DT, 32, 32, 1>(p, st);
}

bool aligned(const void *p, uintptr_t n) { return (uintptr_t)p % n == 0; }

}  // namespace

extern "C" {

size_t moe_gating_topk_grad_workspace(int64_t T, int64_t e)
{
    if (T < 0 || T > INT32_MAX || e < 1 || e > MRR_GATE_MAX_EXPERTS)
        return 0;
    return (size_t)((blocks_for(T) * 2 * e * 4 + 255) / 256 * 256);
}

mrr_status moe_gating_topk_grad_run(const void *grad_y, const void *x, mrr_gate_dtype dt, int64_t T, int64_t e,
                                    int64_t k, const int32_t *expert_idx, const void *bias,
                                    const void *additional_bias, const uint8_t *additional_token_mask,
                                    const float *grad_norm_out, float routed_scaling_factor, float eps,
                                    int64_t norm_type, void *grad_x, void *grad_bias, void *grad_additional_bias,
                                    void *workspace, size_t workspace_bytes, mrr_stream_t stream)
{
    if (dt != MRR_GATE_F16 && dt != MRR_GATE_BF16 && dt != MRR_GATE_F32)
        return MRR_ERR_DTYPE;
    if (norm_type < 0 || norm_type > 2)
        return MRR_ERR_ATTR;
    if (T < 0 || T > INT32_MAX || e < 1 || e > MRR_GATE_MAX_EXPERTS || k < 1 || k > 64 || k > e)
        return MRR_ERR_SHAPE;
    if (T > 0 && (!grad_y || !x || !expert_idx || !grad_x))
        return MRR_ERR_NULL;
    const uintptr_t size = dt == MRR_GATE_F32 ? 4 : 2;
    if (!aligned(grad_y, size) || !aligned(x, size) || !aligned(expert_idx, 4) || !aligned(bias, size) ||
        !aligned(additional_bias, size) || !aligned(grad_norm_out, 4) || !aligned(grad_x, size) ||
        !aligned(grad_bias, size) || !aligned(grad_additional_bias, size))
        return MRR_ERR_ALIGN;
    const bool sums = grad_bias || grad_additional_bias;
    if (sums && T > 0 &&
        (!workspace || !aligned(workspace, 256) || workspace_bytes < moe_gating_topk_grad_workspace(T, e)))
        return MRR_ERR_WORKSPACE;
    // without a mask or an additional bias no row uses one
    const bool masked = additional_bias && additional_token_mask;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (T > 0) {
        Params p;
        memset(&p, 0, sizeof(p));
        p.grad_y = grad_y;
        p.x = x;
        p.bias = bias;
        p.extra_bias = masked ? additional_bias : nullptr;
        p.extra_mask = masked ? additional_token_mask : nullptr;
        p.expert_idx = expert_idx;
        p.grad_norm = grad_norm_out;
        p.grad_x = grad_x;
        p.partial = sums ? static_cast<float *>(workspace) : nullptr;
        p.T = T;
        p.e = (int)e;
        p.k = (int)k;
        p.norm_type = (int)norm_type;
        p.scale = routed_scaling_factor;
        p.eps = eps;
        // groups of four elements, on addresses that are multiples of them
        const bool wide = e % 4 == 0 && aligned(x, 4 * size) && aligned(grad_x, 4 * size) && aligned(grad_norm_out, 16);
        const cudaError_t err = dt == MRR_GATE_F32    ? launch<MOE_F32>(p, wide, st)
                                : dt == MRR_GATE_BF16 ? launch<MOE_BF16>(p, wide, st)
                                                      : launch<MOE_F16>(p, wide, st);
        if (err != cudaSuccess) {
            (void)cudaGetLastError();
            return MRR_ERR_CUDA;
        }
    }
    const int rows = T > 0 ? (int)blocks_for(T) : 0;
    const float *table = static_cast<const float *>(workspace);
    if (grad_bias && launch_column_sum(table, rows, 2 * e, (int)e, dt, grad_bias, st) != cudaSuccess) {
        (void)cudaGetLastError();
        return MRR_ERR_CUDA;
    }
    if (grad_additional_bias &&
        launch_column_sum(table + e, masked ? rows : 0, 2 * e, (int)e, dt, grad_additional_bias, st) != cudaSuccess) {
        (void)cudaGetLastError();
        return MRR_ERR_CUDA;
    }
    return MRR_OK;
}

}  // extern "C"
