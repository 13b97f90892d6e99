// Host entry of the mixture-of-experts layer for a few tokens (include/moe_layer.h): argument checks,
// workspace and shared-memory layout, launch.  The kernel is in moe_layer_kernel.cuh.
#include <atomic>
#include <chrono>

#include "moe_layer_kernel.cuh"

using namespace moe_layer;

namespace {

bool sizes_ok(int64_t T, int64_t H, int64_t E, int64_t I, int64_t k)
{
    return T >= 0 && T <= MOE_LAYER_MAX_TOKENS && H >= 1 && H <= 65536 && I >= 1 && I <= 65536 && E >= 1 &&
           E <= MRR_GATE_MAX_EXPERTS && k >= 1 && k <= 64 && k <= E;
}

constexpr int kDenseTokens = 12;  // more tokens an expert than that, on average: 16-bit weights go to kDense
constexpr int kPairTokens = 4;   // up to so many tokens the second parts of h have columns of their own
constexpr int kMaxGrid = 512;    // blocks; words of the first grid-wide wait, less one

struct Layout {
    size_t waits, part, xh, route_expert, route_weight, x_scale, h_max, h, h_field, split, split_count, bytes;
    int Hp, Ip;
};

Layout layout(int64_t T, int64_t H, int64_t E, int64_t I, int64_t k)
{
    size_t at = mrr_ws::kHeaderBytes;
    auto take = [&at](int64_t bytes) {
        const size_t off = at;
        at += (size_t)mrr_ws::round_up(bytes, 256);
        return off;
    };
    Layout l;
    l.Hp = (int)mrr_ws::round_up(H, 256);   // the products read whole stages, of up to 256 elements
    l.Ip = (int)mrr_ws::round_up(I, 512);   // of x and 512 of h
    l.waits = take(sizeof(Waits) + (kMaxGrid + 1) * 8);
    l.part = take(kMaxParts * T * E * 4);
    l.xh = take(T * l.Hp * 2);
    l.route_expert = take(T * k * 4);
    l.route_weight = take(T * k * 4);
    l.x_scale = take(T * 4);
    l.h_max = take(T * 4);
    l.h = take(2 * T * k * l.Ip * 2);
    l.h_field = take(T * k * (l.Ip / 16));
    const int64_t items = (H + 15) / 16, shares = items > kMaxGrid / 2 ? 0 : items * kMaxSplits < kMaxGrid ? items * kMaxSplits : kMaxGrid;
    l.split = take(shares * T * 16 * 4);
    l.split_count = take(shares ? items * 4 : 0);
    l.bytes = at;
    return l;
}

// 64 bits that no other call of this process has, and that memory holds by chance only: a counter through
// SplitMix64's steps (Steele, Lea, Flood, "Fast splittable pseudorandom number generators", 2014), less the last
unsigned long long fresh_tag()
{
    static std::atomic<unsigned long long> n{
        (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count()};
    unsigned long long z = n.fetch_add(1) * 0x9e3779b97f4a7c15ull;   // a bijection of the counter: odd factors, xor-shifts
    z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
    z ^= z >> 27;
    return z ? z : 1;
}

}  // namespace

extern "C" {

size_t moe_few_token_layer_workspace(int64_t T, int64_t H, int64_t E, int64_t I, int64_t k)
{
    return sizes_ok(T, H, E, I, k) ? layout(T, H, E, I, k).bytes : 0;
}

// moe_few_token_layer_run with another limit on its waits; short_of, where not NULL, is a device word that is 0, or 1 +
// the number of a grid-wide wait that is to expect a block more than there are, or kShortStages, for copies that do
// not count as landed.  What a test calls to see a wait run out.  Not part of the library's interface.
mrr_status moe_few_token_layer_run_waits(const void *x, moe_dtype dt, int64_t T, int64_t H, const void *w_router,
                                         int64_t E, const void *bias, const void *w13, const uint8_t *w13_scales,
                                         const void *w2, const uint8_t *w2_scales, moe_dtype w_dt, int64_t I, int64_t k,
                                         int64_t k_group, int64_t group_count, float routed_scaling_factor, float eps,
                                         int64_t group_select_mode, int64_t norm_type, void *y, float *topk_weight,
                                         int32_t *expert_idx, void *workspace, size_t workspace_bytes,
                                         mrr_stream_t stream, uint64_t wait_ns, const unsigned *short_of)
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
    const Layout l = layout(T, H, E, I, k);
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
    mrr_device::Info info;
    if (!mrr_device::current(info)) {
        (void)cudaGetLastError();
        return MRR_ERR_CUDA;
    }
    const int grid = info.sms < kMaxGrid ? info.sms : kMaxGrid;
    Params p{};
    p.x = x, p.wr = w_router, p.bias = bias, p.w13 = w13, p.w2 = w2, p.w13_s = w13_scales, p.w2_s = w2_scales;
    p.T = (int)T, p.H = (int)H, p.E = (int)E, p.I = (int)I, p.k = (int)k;
    p.k_group = (int)k_group, p.group_count = (int)group_count;
    p.select_mode = (int)group_select_mode, p.norm_type = (int)norm_type;
    p.rsf = routed_scaling_factor, p.eps = eps;
    p.y = y, p.topk_weight = topk_weight, p.expert_idx = expert_idx;
    p.status = reinterpret_cast<uint32_t *>(ws);
    p.waits = reinterpret_cast<Waits *>(ws + l.waits);
    p.tag = fresh_tag();
    p.wait_ns = wait_ns, p.short_of = short_of;
    p.part = reinterpret_cast<float *>(ws + l.part);
    p.xh = reinterpret_cast<uint16_t *>(ws + l.xh);
    p.route_expert = reinterpret_cast<int *>(ws + l.route_expert);
    p.route_weight = reinterpret_cast<float *>(ws + l.route_weight);
    p.x_scale = reinterpret_cast<float *>(ws + l.x_scale);
    p.h_max = reinterpret_cast<uint32_t *>(ws + l.h_max);
    p.h = reinterpret_cast<uint16_t *>(ws + l.h);
    p.pairs = T <= kPairTokens;
    p.h_field = ws + l.h_field;
    p.split = reinterpret_cast<float *>(ws + l.split);
    p.split_count = reinterpret_cast<unsigned *>(ws + l.split_count);
    p.Hp = l.Hp, p.Ip = l.Ip;
    // the router's 16-expert tiles, split over H until the blocks have one each
    const int64_t tiles = (E + 15) / 16, chunks = (H + 127) / 128;
    int64_t parts = grid / tiles;
    parts = parts < 1 ? 1 : parts > kMaxParts ? kMaxParts : parts;
    p.kparts = (int)(parts < chunks ? parts : chunks);
    auto wide = [](const void *a, int64_t row_bytes, int by) { return (uintptr_t)a % by == 0 && row_bytes % by == 0; };
    p.x_wide = wide(x, 2 * H, 16);
    p.wr_wide = wide(w_router, 2 * H, 16);
    p.w13_wide = wide(w13, mx ? H / 2 : 2 * H, 16);
    p.w2_wide = wide(w2, mx ? I / 2 : 2 * I, 16);
    if (p.w13_wide && p.w2_wide &&
        (!tc::make_map(&p.w13_map, w13, E * 2 * I, mx ? H / 2 : 2 * H, 16) ||
         !tc::make_map(&p.w2_map, w2, E * H, mx ? I / 2 : 2 * I, 16)))
        return MRR_ERR_CUDA;
    p.s13_wide = mx && wide(w13_scales, scale_row_bytes(H), 8);
    p.s2_wide = mx && wide(w2_scales, scale_row_bytes(I), 8);
    const int regime = T <= 8 ? kFew : !mx && T * k > kDenseTokens * E ? kDense : kSpread;
    // shared memory: the rings (before them, the routing's scratch), the joins, who goes where
    // active experts, counted as often as they are streamed
    const int64_t n = T * k, active = (n < E ? n : E) + (T > 8 ? n / (8 * tiles_for(mx, regime)) : 0);
    const bool rows_wide = p.w13_wide && p.w2_wide;
    const int warps = warps_of(mx, rows_wide, regime), stages = stages_of(mx, rows_wide, regime);
    int64_t at = (int64_t)warps * stages * stage_of(rows_wide);
    const int64_t keys = ((T > 8 ? 1 : T) * 2 * E + E) * 4, places = 2 * (E + n);
    p.sm_scratch = (int)mrr_ws::round_up(2 * n, 16);
    const int64_t scratch = p.sm_scratch + (keys > places ? keys : places);
    at = at > scratch ? mrr_ws::round_up(at, 16) : mrr_ws::round_up(scratch, 16);
    auto take = [&at](int64_t bytes) {
        const int64_t off = at;
        at += mrr_ws::round_up(bytes, 16);
        return (int)off;
    };
    p.sm_scales = mx ? take(warps * stages * kStageScales) : 0;
    p.sm_bar = take(warps * stages * 8);
    const int64_t joins = 2 * warps * 256 * 4, sums = T > 8 ? warps * T * 17 * 4 : 0;   // of up and down: not at once
    p.sm_red = take(joins > sums ? joins : sums);
    p.sm_weight = take((T > 8 ? k : n) * 4);
    p.sm_act = take(active * 2);
    p.sm_start = take((active + 1) * 2);
    p.sm_cols = take(T > 8 ? n * 2 : active * 16);
    p.sm_tokens = T > 8 ? take(n) : 0;
    p.sm_count = take(16);
    if (at > info.smem_max)
        return MRR_ERR_CUDA;
    // y's rows in items of 16: blocks share them where there are two blocks or more to each, and work for them
    const int64_t down_items = (H + 15) / 16, down_chunks = (I + (mx ? 511 : 127)) / (mx ? 512 : 128);
    const bool split = 2 * down_items <= grid && active * down_chunks >= 4 * warps;
    Launch *launch = dt == MOE_BF16 ? (split ? launch_bf16_split : launch_bf16) : (split ? launch_f16_split : launch_f16);
    const cudaError_t err = launch(p, mx, regime, info, grid, (size_t)at, s);
    if (err != cudaSuccess) {
        (void)cudaGetLastError();
        return MRR_ERR_CUDA;
    }
    return MRR_OK;
}

mrr_status moe_few_token_layer_run(const void *x, moe_dtype dt, int64_t T, int64_t H, const void *w_router, int64_t E,
                                   const void *bias, const void *w13, const uint8_t *w13_scales, const void *w2,
                                   const uint8_t *w2_scales, moe_dtype w_dt, int64_t I, int64_t k, int64_t k_group,
                                   int64_t group_count, float routed_scaling_factor, float eps,
                                   int64_t group_select_mode, int64_t norm_type, void *y, float *topk_weight,
                                   int32_t *expert_idx, void *workspace, size_t workspace_bytes, mrr_stream_t stream)
{
    return moe_few_token_layer_run_waits(x, dt, T, H, w_router, E, bias, w13, w13_scales, w2, w2_scales, w_dt, I, k, k_group,
                                         group_count, routed_scaling_factor, eps, group_select_mode, norm_type, y,
                                         topk_weight, expert_idx, workspace, workspace_bytes, stream, kWaitLimitNs, nullptr);
}

}  // extern "C"
