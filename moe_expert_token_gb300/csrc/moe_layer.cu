// The whole mixture-of-experts layer for a few tokens (include/moe_layer.h).
#include <math.h>

#include "moe_layer.h"
#include "mrr_gating.h"
#include "mx.cuh"
#include "ws_layout.h"

using namespace moe_mx;

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 256, kWarps = kThreads / 32;

struct Params {
    const void *x, *wr, *bias, *w13, *w2;
    const uint8_t *w13_s, *w2_s;
    int T, H, E, I, k, k_group, group_count, select_mode, norm_type;
    float rsf, eps;
    void *y;
    float *topk_weight;
    int *expert_idx;
    uint32_t *status;
    float *logits, *weight, *h;   // [T, E], [T, k], [T, k, I]
    int *expert;                  // [T, k]
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// element k of row `row` of weights [rows, K]
template <int WDT>
__device__ __forceinline__ float weight_at(const void *w, const uint8_t *s, int64_t row, int K, int k)
{
    if (WDT == MOE_MXFP4) {
        const uint32_t q = __ldg(static_cast<const uint8_t *>(w) + row * (K / 2) + k / 2);
        return decode1(k % 2 ? q >> 4 : q) * e8m0_value(__ldg(s + row * scale_row_bytes(K) + k / 32));
    }
    return load1<WDT == MOE_MXFP4 ? MOE_F32 : WDT>(w, row * K + k);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) router_simple(Params p)
{
    const int u = blockIdx.x * kWarps + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (blockIdx.x == 0 && threadIdx.x < 2)
        p.status[threadIdx.x] = 0;
    if (u >= p.T * p.E)
        return;
    const int t = u / p.E, e = u % p.E;
    float a = 0.f;
    for (int i = lane; i < p.H; i += 32)
        a = fmaf(load1<DT>(p.x, (int64_t)t * p.H + i), load1<DT>(p.wr, (int64_t)e * p.H + i), a);
    a = warp_sum(a);
    if (lane == 0)
        p.logits[u] = a;
}

// one warp a token; scores in shared memory
template <int DT>
__global__ void __launch_bounds__(32) gate_simple(Params p)
{
    __shared__ float score[MRR_GATE_MAX_EXPERTS], group[MRR_GATE_MAX_EXPERTS];
    __shared__ uint8_t live[MRR_GATE_MAX_EXPERTS];
    const int t = blockIdx.x, lane = threadIdx.x, size = p.E / p.group_count;
    const float *z = p.logits + (int64_t)t * p.E;
    float mx = -INFINITY, sum = 0.f;
    for (int e = lane; e < p.E; e += 32)
        mx = fmaxf(mx, z[e]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    for (int e = lane; e < p.E; e += 32)
        sum += expf(z[e] - mx);
    sum = warp_sum(sum);
    for (int e = lane; e < p.E; e += 32) {
        float s;
        if (p.norm_type == 0)
            s = expf(z[e] - mx) / sum;
        else if (p.norm_type == 1)
            s = 1.f / (1.f + expf(-z[e]));
        else
            s = z[e] > 20.f ? z[e] + log1pf(expf(-z[e])) : log1pf(expf(z[e]));
        score[e] = p.bias ? s + load1<DT>(p.bias, e) : s;
        live[e] = 1;
    }
    __syncwarp();
    // the best of what `ok` admits: larger value, then lower index; a NaN ranks below everything
    auto best = [&](const float *v, int n, auto ok) {
        float bv = -INFINITY;
        int bi = n;
        for (int e = lane; e < n; e += 32)
            if (ok(e) && (bi == n || v[e] > bv || (bv != bv && v[e] == v[e]))) {
                bv = v[e];
                bi = e;
            }
        if (bv != bv)
            bv = -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float ov = __shfl_xor_sync(kFull, bv, o);
            const int oi = __shfl_xor_sync(kFull, bi, o);
            if (oi < n && (bi == n || ov > bv || (ov == bv && oi < bi))) {
                bv = ov;
                bi = oi;
            }
        }
        return bi;
    };
    if (p.group_count > 1 && p.k_group < p.group_count) {
        for (int g = lane; g < p.group_count; g += 32) {
            float a = -INFINITY, b = -INFINITY;
            for (int e = g * size; e < (g + 1) * size; ++e) {
                const float s = score[e];
                if (s > a)
                    b = a, a = s;
                else if (s > b)
                    b = s;
            }
            group[g] = p.select_mode == 1 ? a + b : a;
        }
        for (int e = lane; e < p.E; e += 32)
            live[e] = 0;
        __syncwarp();
        for (int i = 0; i < p.k_group; ++i) {
            const int g = best(group, p.group_count, [&](int e) { return live[e * size] == 0; });
            __syncwarp();
            for (int e = g * size + lane; e < (g + 1) * size; e += 32)
                live[e] = 1;
            __syncwarp();
        }
    }
    float total = 0.f;
    for (int i = 0; i < p.k; ++i) {
        const int e = best(score, p.E, [&](int e) { return live[e] != 0; });
        __syncwarp();
        if (lane == 0) {
            live[e] = 0;
            p.expert[t * p.k + i] = e;
        }
        total += score[e];
        __syncwarp();
    }
    for (int i = lane; i < p.k; i += 32) {
        const int e = p.expert[t * p.k + i];
        const float w = score[e] / (total + p.eps) * p.rsf;
        p.weight[t * p.k + i] = w;
        if (p.topk_weight)
            p.topk_weight[t * p.k + i] = w;
        if (p.expert_idx)
            p.expert_idx[t * p.k + i] = e;
    }
}

template <int DT, int WDT>
__global__ void __launch_bounds__(kThreads) up_simple(Params p)
{
    const int64_t u = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (u >= (int64_t)p.T * p.k * p.I)
        return;
    const int a = (int)(u / p.I), i = (int)(u % p.I), t = a / p.k;
    const int64_t row = (int64_t)p.expert[a] * 2 * p.I + i;
    float g = 0.f, up = 0.f;
    for (int c = lane; c < p.H; c += 32) {
        const float x = load1<DT>(p.x, (int64_t)t * p.H + c);
        g = fmaf(x, weight_at<WDT>(p.w13, p.w13_s, row, p.H, c), g);
        up = fmaf(x, weight_at<WDT>(p.w13, p.w13_s, row + p.I, p.H, c), up);
    }
    g = warp_sum(g);
    up = warp_sum(up);
    if (lane == 0)
        p.h[u] = g / (1.f + expf(-g)) * up;
}

template <int DT, int WDT>
__global__ void __launch_bounds__(kThreads) down_simple(Params p)
{
    const int64_t u = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (u >= (int64_t)p.T * p.H)
        return;
    const int t = (int)(u / p.H), n = (int)(u % p.H);
    float y = 0.f;
    for (int j = 0; j < p.k; ++j) {
        const int a = t * p.k + j;
        const int64_t row = (int64_t)p.expert[a] * p.H + n;
        float s = 0.f;
        for (int c = lane; c < p.I; c += 32)
            s = fmaf(p.h[(int64_t)a * p.I + c], weight_at<WDT>(p.w2, p.w2_s, row, p.I, c), s);
        y = fmaf(p.weight[a], warp_sum(s), y);
    }
    if (lane == 0)
        store1<DT>(p.y, u, y);
}

template <int DT, int WDT>
void launch(const Params &p, cudaStream_t s)
{
    auto grid = [](int64_t units) { return (unsigned)((units + kWarps - 1) / kWarps); };
    router_simple<DT><<<grid((int64_t)p.T * p.E), kThreads, 0, s>>>(p);
    gate_simple<DT><<<p.T, 32, 0, s>>>(p);
    up_simple<DT, WDT><<<grid((int64_t)p.T * p.k * p.I), kThreads, 0, s>>>(p);
    down_simple<DT, WDT><<<grid((int64_t)p.T * p.H), kThreads, 0, s>>>(p);
}

bool sizes_ok(int64_t T, int64_t H, int64_t E, int64_t I, int64_t k)
{
    return T >= 0 && T <= MOE_LAYER_MAX_TOKENS && H >= 1 && H <= 65536 && I >= 1 && I <= 65536 && E >= 1 &&
           E <= MRR_GATE_MAX_EXPERTS && k >= 1 && k <= 64 && k <= E;
}

struct Layout {
    size_t logits, weight, expert, h, bytes;
};

Layout layout(int64_t T, int64_t E, int64_t I, int64_t k)
{
    size_t at = mrr_ws::kHeaderBytes;
    auto take = [&at](int64_t words) {
        const size_t off = at;
        at += (size_t)mrr_ws::round_up(4 * words, 256);
        return off;
    };
    Layout l;
    l.logits = take(T * E);
    l.weight = take(T * k);
    l.expert = take(T * k);
    l.h = take(T * k * I);
    l.bytes = at;
    return l;
}

}  // namespace

extern "C" {

size_t moe_few_token_layer_workspace(int64_t T, int64_t H, int64_t E, int64_t I, int64_t k)
{
    return sizes_ok(T, H, E, I, k) ? layout(T, E, I, k).bytes : 0;
}

mrr_status moe_few_token_layer_run(const void *x, moe_dtype dt, int64_t T, int64_t H, const void *w_router, int64_t E,
                                   const void *bias, const void *w13, const uint8_t *w13_scales, const void *w2,
                                   const uint8_t *w2_scales, moe_dtype w_dt, int64_t I, int64_t k, int64_t k_group,
                                   int64_t group_count, float routed_scaling_factor, float eps,
                                   int64_t group_select_mode, int64_t norm_type, void *y, float *topk_weight,
                                   int32_t *expert_idx, void *workspace, size_t workspace_bytes, mrr_stream_t stream)
{
    if ((dt != MOE_F16 && dt != MOE_BF16) || (w_dt != dt && w_dt != MOE_MXFP4))
        return MRR_ERR_DTYPE;
    if (group_select_mode < 0 || group_select_mode > 1 || norm_type < 0 || norm_type > 2)
        return MRR_ERR_ATTR;
    const bool mx = w_dt == MOE_MXFP4;
    if (!sizes_ok(T, H, E, I, k) || (mx && (H % 2 || I % 2)))
        return MRR_ERR_SHAPE;
    if (group_count < 1 || k_group < 1 || k_group > group_count || E % group_count ||
        k > (E / group_count) * k_group || (group_select_mode == 1 && E / group_count < 2))
        return MRR_ERR_SHAPE;
    if (T > 0 && (!x || !w_router || !w13 || !w2 || !y || (mx && (!w13_scales || !w2_scales))))
        return MRR_ERR_NULL;
    if ((uintptr_t)x % 2 || (uintptr_t)w_router % 2 || (uintptr_t)bias % 2 || (uintptr_t)y % 2 ||
        (!mx && ((uintptr_t)w13 % 2 || (uintptr_t)w2 % 2)) || (uintptr_t)topk_weight % 4 || (uintptr_t)expert_idx % 4)
        return MRR_ERR_ALIGN;
    const Layout l = layout(T, E, I, k);
    if (!workspace || (uintptr_t)workspace % 256 || workspace_bytes < l.bytes)
        return MRR_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (T == 0) {
        if (cudaMemsetAsync(ws, 0, 8, s) != cudaSuccess) {
            (void)cudaGetLastError();
            return MRR_ERR_CUDA;
        }
        return MRR_OK;
    }
    Params p{};
    p.x = x, p.wr = w_router, p.bias = bias, p.w13 = w13, p.w2 = w2, p.w13_s = w13_scales, p.w2_s = w2_scales;
    p.T = (int)T, p.H = (int)H, p.E = (int)E, p.I = (int)I, p.k = (int)k;
    p.k_group = (int)k_group, p.group_count = (int)group_count;
    p.select_mode = (int)group_select_mode, p.norm_type = (int)norm_type;
    p.rsf = routed_scaling_factor, p.eps = eps;
    p.y = y, p.topk_weight = topk_weight, p.expert_idx = expert_idx;
    p.status = reinterpret_cast<uint32_t *>(ws);
    p.logits = reinterpret_cast<float *>(ws + l.logits);
    p.weight = reinterpret_cast<float *>(ws + l.weight);
    p.expert = reinterpret_cast<int *>(ws + l.expert);
    p.h = reinterpret_cast<float *>(ws + l.h);
    if (dt == MOE_F16)
        mx ? launch<MOE_F16, MOE_MXFP4>(p, s) : launch<MOE_F16, MOE_F16>(p, s);
    else
        mx ? launch<MOE_BF16, MOE_MXFP4>(p, s) : launch<MOE_BF16, MOE_BF16>(p, s);
    return cudaGetLastError() == cudaSuccess ? MRR_OK : MRR_ERR_CUDA;
}

}  // extern "C"
