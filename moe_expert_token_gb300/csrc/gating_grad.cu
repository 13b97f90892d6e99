// The gradient of the MoE gating top-k op (include/mrr_gating.h, mrr_gating_topk_grad_run).
//
// Scores that stand alone (sigmoid, softplus) without a gradient of the normalised output: grad_x is zero but for
// the k chosen experts (gating_grad_chosen).  A group of lanes has a token, a lane a chosen expert, so several tokens share
// a warp; x is read where it is needed, and the row of zeros is written ahead of the k values.  Else every
// element of x has a share (gating_grad_dense): a warp has a token, each lane every 32nd expert, and the chosen
// experts' shares are added into a row in shared memory.  Each element is read or written once with one or
// two exponentials between: for the usual sizes (16384 rows of 256 in 16 bits, 8 to 17 MB) launches and the latency of a
// row count for as much as HBM.
//
// The gradient of the biases is a sum over rows: warps hold sums of their own while the block goes from row to row,
// each block leaves one row of partial sums, and a second launch adds those in order.
#include <atomic>
#include <string.h>

#include "column_sum.cuh"
#include "device_info.h"
#include "mrr_gating.h"

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

// LANES lanes a token (k <= LANES; 32 lanes: two slots each).  sums: [2][e] of each warp, where bias gradients are asked for.
template <int DT, int LANES>
__global__ void __launch_bounds__(32 * kWarps) gating_grad_chosen(Params p)
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
        float g[kSlots], x[kSlots], d[kSlots], sum = 0.0f, inner = 0.0f;
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
        for (int h = 0; h < kSlots; ++h) {
            x[h] = idx[h] >= 0 ? load1<DT>(p.x, t * p.e + idx[h]) : 0.0f;
            float s = 0.0f;
            if (idx[h] >= 0)
                s = score_of(p.norm_type, x[h], 0.0f, 1.0f) + (bias ? load1<DT>(bias, idx[h]) : 0.0f);
            sum += s;
            inner = fmaf(g[h], s, inner);
        }
        clear<DT == MOE_F32 ? 4 : 2>(p.grad_x, t0 * p.e, min((int64_t)kTokens, p.T - t0) * p.e, lane, 32);
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
            d[h] = factor * (g[h] - inner);
        // an expert that a token has twice (hash routing): its first slot gets the sum, in the order of the slots
        bool twice = false;
#pragma unroll
        for (int h = 0; h < kSlots; ++h) {
            const uint32_t group = LANES == 32 ? kFull : ((1u << LANES) - 1) << (of_warp * LANES);
            const uint32_t same = __match_any_sync(kFull, idx[h]) & group;
            twice |= idx[h] >= 0 && __popc(same) > 1;
            if (kSlots == 2 && h == 1)
                twice = twice || p.k > 32;   // the two halves are not compared here
        }
        if (__any_sync(kFull, twice)) {
            float all[kSlots];
            bool first[kSlots];
#pragma unroll
            for (int h = 0; h < kSlots; ++h)
                all[h] = 0.0f, first[h] = true;
#pragma unroll
            for (int o = 0; o < kSlots; ++o)
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
                    idx[h] = -1;
            }
        }
        __syncwarp();   // the zeros are written
#pragma unroll
        for (int h = 0; h < kSlots; ++h)
            if (idx[h] >= 0)
                store1<DT>(p.grad_x, t * p.e + idx[h], d[h] * slope_of(p.norm_type, x[h]));
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

template <int DT, int VPL>
__global__ void __launch_bounds__(32 * kWarps) gating_grad_dense(Params p)
{
    extern __shared__ float rows[];   // [kWarps][e]
    mrr::grid_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    float *ds = rows + warp * p.e;
    float acc[VPL], extra_acc[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        acc[i] = extra_acc[i] = 0.0f;
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < p.T; t += (int64_t)gridDim.x * kWarps) {
        float x[VPL];
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int at = 32 * i + lane;
            x[i] = at < p.e ? load1<DT>(p.x, t * p.e + at) : -INFINITY;
            top = fmaxf(top, x[i]);
            if (at < p.e)
                ds[at] = p.grad_norm ? __ldg(p.grad_norm + t * p.e + at) : 0.0f;
        }
        float total = 1.0f;
        if (p.norm_type == 0) {
#pragma unroll
            for (int d = 16; d > 0; d /= 2)
                top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                x[i] = 32 * i + lane < p.e ? expf(x[i] - top) : 0.0f;   // the scores, but for their sum
                total += x[i];
            }
            total = warp_sum(total);
        }
        const bool extra = p.extra_mask && p.extra_bias && p.extra_mask[t] != 0;
        const void *bias = extra ? p.extra_bias : p.bias;
        // up to two slots a lane
        int idx[2];
        float g[2], s[2], sum = 0.0f, inner = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = 32 * h + lane;
            idx[h] = j < p.k ? __ldg(p.expert_idx + t * p.k + j) : -1;
            if (idx[h] >= p.e)
                idx[h] = -1;
            g[h] = s[h] = 0.0f;
            if (idx[h] >= 0) {
                g[h] = load1<DT>(p.grad_y, t * p.k + j);
                s[h] = score_of(p.norm_type, load1<DT>(p.x, t * p.e + idx[h]), top, total);
                if (bias)
                    s[h] += load1<DT>(bias, idx[h]);
            }
            sum += s[h];
            inner = fmaf(g[h], s[h], inner);
        }
        sum = warp_sum(sum) + p.eps;
        inner = warp_sum(inner) / sum;
        const float factor = p.scale / sum;
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (32 * h >= p.k)
                break;
            const float d = factor * (g[h] - inner);
            const uint32_t same = __match_any_sync(kFull, idx[h]);
            const bool twice = __any_sync(kFull, idx[h] >= 0 && __popc(same) > 1);
            if (!twice) {
                if (idx[h] >= 0)
                    ds[idx[h]] += d;
            } else {   // an expert twice in one row (hash routing): one lane after the other
                for (int l = 0; l < 32; ++l) {
                    if (l == lane && idx[h] >= 0)
                        ds[idx[h]] += d;
                    __syncwarp();
                }
            }
            __syncwarp();
        }
        float dot = 0.0f;
        if (p.norm_type == 0) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int at = 32 * i + lane;
                x[i] /= total;
                dot = fmaf(x[i], at < p.e ? ds[at] : 0.0f, dot);
            }
            dot = warp_sum(dot);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int at = 32 * i + lane;
            if (at >= p.e)
                continue;
            const float d = ds[at];
            float out;
            if (p.norm_type == 0)
                out = x[i] * (d - dot);
            else
                out = d * slope_of(p.norm_type, x[i]);
            store1<DT>(p.grad_x, t * p.e + at, out);
            if (extra)
                extra_acc[i] += d;
            else
                acc[i] += d;
        }
        __syncwarp();
    }
    if (!p.partial)
        return;
    // the warps' sums, in order
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (which && !p.extra_mask)
            break;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (32 * i + lane < p.e)
                ds[32 * i + lane] = which ? extra_acc[i] : acc[i];
        __syncthreads();
        for (int at = threadIdx.x; at < p.e; at += 32 * kWarps) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                s += rows[w * p.e + at];
            p.partial[((int64_t)blockIdx.x * 2 + which) * p.e + at] = s;
        }
    }
}

int64_t blocks_for(int64_t T)
{
    const int64_t blocks = (T + kWarps - 1) / kWarps;
    return blocks < kMaxBlocks ? blocks : kMaxBlocks;
}

template <int DT, int LANES>
cudaError_t launch_chosen(const Params &p, cudaStream_t st)
{
    static std::atomic<uint64_t> done;
    mrr_device::Info info;
    if (!mrr_device::current(info))
        return cudaErrorUnknown;
    const int smem = p.partial ? kWarps * (p.extra_mask ? 2 : 1) * p.e * 4 : 0;   // up to 64 KB
    const cudaError_t err = mrr_device::allow_smem(gating_grad_chosen<DT, LANES>, info, done);
    if (err != cudaSuccess)
        return err;
    gating_grad_chosen<DT, LANES><<<(unsigned)blocks_for(p.T), 32 * kWarps, smem, st>>>(p);
    return cudaGetLastError();
}

template <int DT>
cudaError_t launch(const Params &p, cudaStream_t st)
{
    if (p.norm_type != 0 && !p.grad_norm)
        return p.k <= 8 ? launch_chosen<DT, 8>(p, st) : p.k <= 16 ? launch_chosen<DT, 16>(p, st) : launch_chosen<DT, 32>(p, st);
    const int smem = kWarps * p.e * 4, per = (p.e + 31) / 32;
    auto kernel = per <= 2    ? gating_grad_dense<DT, 2>
                  : per <= 4  ? gating_grad_dense<DT, 4>
                  : per <= 8  ? gating_grad_dense<DT, 8>
                  : per <= 16 ? gating_grad_dense<DT, 16> : gating_grad_dense<DT, 32>;
    kernel<<<(unsigned)blocks_for(p.T), 32 * kWarps, smem, st>>>(p);
    return cudaGetLastError();
}

bool aligned(const void *p, uintptr_t n) { return (uintptr_t)p % n == 0; }

}  // namespace

extern "C" {

size_t mrr_gating_topk_grad_workspace(int64_t T, int64_t e)
{
    if (T < 0 || T > INT32_MAX || e < 1 || e > MRR_GATE_MAX_EXPERTS)
        return 0;
    return (size_t)((blocks_for(T) * 2 * e * 4 + 255) / 256 * 256);
}

mrr_status mrr_gating_topk_grad_run(const void *grad_y, const void *x, mrr_gate_dtype dt, int64_t T, int64_t e,
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
        (!workspace || !aligned(workspace, 256) || workspace_bytes < mrr_gating_topk_grad_workspace(T, e)))
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
        const cudaError_t err = dt == MRR_GATE_F32    ? launch<MOE_F32>(p, st)
                                : dt == MRR_GATE_BF16 ? launch<MOE_BF16>(p, st)
                                                      : launch<MOE_F16>(p, st);
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
