// The kernel of the mixture-of-experts layer for a few tokens (include/moe_layer.h), for GB300
// (sm_103a).  moe_layer_{bf16,f16}[_split].cu instantiate it, moe_layer.cu holds the host entry.
//
//   logits = x w_router^T;  experts, weights = gating(logits)
//   h[a, i] = weight[a] silu(w13[e, i] . x) (w13[e, I + i] . x)      for each assignment a = (token, expert)
//   y[t, n] = sum over t's assignments of w2[e, n] . h[a]
//
// What it has to move is the chosen experts' weights, each read once; for a few tokens that is all
// that counts, so the layer is one persistent kernel (one block for each SM, launched
// cooperatively) that streams weights without a pause:
//  * Weights are rows of a 16-row matrix-instruction tile, tokens its 8 columns (m16n8k16, float32
//    sums).  A tile of 8 columns costs no more for one token than for eight, and the tensor pipe
//    is idle most of the time: the rate that matters is that of the loads.
//  * Each warp streams its own share of the K axis through a private ring of kStages 4 KB stages in
//    shared memory.  A stage is two slabs of 16 rows x 128 bytes, each one tiled bulk copy issued by
//    one lane (thread copies of 16 bytes, with their addresses, were most of the instructions that
//    a stage cost; they bring rows that are not aligned to 16 bytes).  The ring runs on across items, and from the up product into the down product:
//    the down weights of the first items are in flight while the grid waits for h.
//  * A lane's 16-byte piece of a row feeds two matrix instructions: the order of k inside a group of
//    32 is free as long as both operands share it, so lane (g, t) holds elements 8t .. 8t+7.
//  * The grid waits twice: for the logits, and for h.  Between them every block computes the
//    routing of all tokens for itself, which costs less than a third wait; with more than 8 tokens
//    each token's is one block's work, and there is one.
//  * Up product: an item is 16 gate rows and the 16 up rows that belong to them, K split over the
//    warps, joined in shared memory, or all of K by one warp; SwiGLU and the routing weight are
//    applied to the sums, in float32.
//  * Down product: an item is 16 output rows for all tokens; the warps split (expert, K) pairs, and where
//    there are few items, several blocks do.
// Measured, with x and the weights from HBM: 1 token, 64 experts of 7168 x 2048 in bfloat16, top 8 (706 MB)
// 118 us, 6.0 TB/s; 48 tokens (5.64 GB) 928 us, 6.1 TB/s; 7 tokens, 60 experts of 2056 x 1400 in float16, top
// 6 (0.54 GB) 104 us, 5.2 TB/s; 4 tokens, 256 MXFP4 experts of 7168 x 2048, top 8 (0.72 GB) 182 us, 4.0 TB/s,
// bound by the instructions that unpack; 1 token, 8 experts of 1024 x 512 (6 MB) 16 us, bound by the
// latency of three phases that wait for one another.
// With up to 8 tokens the columns are the tokens themselves and the down product adds up all
// experts in registers; with more, an expert's columns are the tokens that chose it, and each
// warp adds them to its own sums in shared memory.  The order of every sum goes by the sizes and by how many
// experts the tokens reach: the same inputs give the same bits, but a token's last bits may differ with the
// tokens beside it.
#pragma once

#include <math.h>

#include "device_info.h"
#include "moe_layer.h"
#include "mrr_gating.h"
#include "mx.cuh"
#include "ptx.cuh"
#include "tc.cuh"
#include "ws_layout.h"

namespace moe_layer {

using namespace moe_mx;

constexpr uint32_t kFull = 0xffffffffu;
// How the columns of the matrix instructions, in tiles of 8, are used.
//  * kFew, up to 8 tokens: one tile, whose columns are the tokens.
//  * kSpread: the columns are the tokens that chose the expert, in up to 4 tiles, two of them loaded ahead;
//    one tile for MXFP4, whose unpacking needs the registers.  An expert with more tokens than that is
//    streamed once for each tileful (the second time from L2: both run at about the same time).
//  * kDense, 16-bit weights of experts with many tokens: all 4 tiles are loaded ahead, which takes all
//    registers.  48 tokens, 16 experts of 7168 x 2048, 24 tokens an expert: 474 -> 402 us; 64 tokens, 16
//    experts of 2048 x 1408, 32 an expert: 224 -> 175; 6 to 16 an expert: the same to 2 % slower.
//    (For MXFP4, in half as long steps and with 8 warps: 16 tokens an expert 139 -> 162, 24 the same.)
enum Regime { kFew, kSpread, kDense };
__host__ __device__ constexpr int tiles_for(bool mx, int regime) { return regime == kFew || mx ? 1 : 4; }
// Warps of a block and stages of a warp's ring.  Unpacking 4-bit weights is bound by how many
// instructions are ready, so MXFP4 has 12 warps (as many as registers allow) with shorter rings (4 tokens,
// 256 experts of 7168 x 2048: 182 us, with 8 warps 201); the 16-bit types stream at the memory's rate with 8.
// Rows that tiled copies cannot take (narrow) cost instructions too, and have 12 where registers and
// memory allow (7 tokens, 60 experts of 2055 x 1399: 151 us, with 8 warps 168).
__host__ __device__ constexpr int warps_of(bool mx, bool wide, int regime)
{
    return wide ? (mx ? 12 : 8) : regime == kFew ? 12 : 8;
}
__host__ __device__ constexpr int stages_of(bool mx, bool wide, int regime) { return warps_of(mx, wide, regime) == 12 ? 3 : 4; }
// Bytes of a stage's row, and of a stage: two slabs of 16 rows.  Narrow rows come as nine aligned 16-byte
// pieces and are shifted into place when they are read.
__host__ __device__ constexpr int pitch_of(bool wide) { return wide ? 128 : 144; }
__host__ __device__ constexpr int stage_of(bool wide) { return 2 * 16 * pitch_of(wide); }
constexpr int kMaxParts = 16;                    // most shares of H the logits are split into
constexpr int kMaxSplits = 16;                   // most blocks that share a down item
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr unsigned kShortStages = 4;

struct Params {
    const void *x, *wr, *bias, *w13, *w2;
    const uint8_t *w13_s, *w2_s;
    int T, H, E, I, k, k_group, group_count, select_mode, norm_type;
    float rsf, eps;
    void *y;
    float *topk_weight;
    int *expert_idx;
    // workspace
    uint32_t *status;
    struct Waits *waits;          // see grid_wait
    unsigned long long tag;
    uint64_t wait_ns;             // limit of each wait
    const unsigned *short_of;     // null, or (tests that let a wait run out) a word: 1 + the grid-wide wait that expects a
                                  // block more, or kShortStages: the stages' barriers expect an arrival more
    float *part;                  // [kparts][T][E]
    uint16_t *xh;                 // [T][Hp]: x's rows as the products take them
    int *route_expert;            // [T][k], with more than 8 tokens
    float *route_weight;
    float *x_scale;               // [T]: what undoes their scaling
    uint32_t *h_max;              // [T]: float bits of the largest |h| of the token
    // h as the sum of two 16-bit parts, so that y is rounded once, at its end: with one part y's error was 1.4 times
    // that.  Up to 4 tokens (pairs) the second parts take the four columns of the down product that the tokens
    // leave; with more they are a second product with the same weights, which costs 3 % of a layer for 48 tokens,
    // 4 % for 7, and 21 % where an expert has 24 tokens.  With MXFP4 weights and y in bfloat16 more than 4 tokens
    // have one (float16) part, see kParts.  An element's parts lie 16 bytes apart, so that one load brings both.
    uint16_t *h;                  // [T k][Ip / 8][parts][8]
    int pairs;
    float *split;                 // [splits][H / 16, rounded up][T][16]: y's shares where blocks split its sums
    unsigned *split_count;        // [H / 16, rounded up]: shares that are there
    uint8_t *h_field;             // [T k][Ip / 16]: exponent of the power of two each tile of h carries (float16)
    int Hp, Ip, kparts;
    int x_wide, wr_wide;              // 16-byte loads possible
    int w13_wide, w2_wide;            // rows are 16-byte aligned: tiled copies possible
    int s13_wide, s2_wide;            // scale rows are 8-byte aligned
    CUtensorMap w13_map, w2_map;      // rows of bytes, boxes of 128 bytes x 16 rows, 128-byte swizzle
    // dynamic shared memory, byte offsets
    int sm_scales, sm_bar, sm_red, sm_scratch, sm_weight, sm_act, sm_start, sm_cols, sm_tokens, sm_count;
};

constexpr int kStageScales = 256;

template <int DT>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    if (DT == MOE_BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// an asynchronous copy of 8 bytes: the first `bytes` of them are read, the rest zeros
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// of 16 bytes
__device__ __forceinline__ void copy16(uint32_t dst, uintptr_t src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// the first `bytes` of them are read, the rest zeros
__device__ __forceinline__ void copy16(uint32_t dst, uintptr_t src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// this thread arrives on `bar` once its copies so far have landed
__device__ __forceinline__ void copies_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// The power of two that takes the float with bits `amax` into [2^14, 2^15), so that it and all
// smaller ones fit float16: its exponent field.  1 for an infinite or NaN amax; the largest for 0.
__device__ __forceinline__ uint32_t f16_scale_field(uint32_t amax)
{
    const int field = (int)(amax >> 23);
    return field == 255 ? 127u : (uint32_t)min(268 - field, 253);   // field <= 254: at least 14
}

// v rounded to 16 bits (an infinity or NaN: 0, so that v less this is v)
template <int DT>
__device__ __forceinline__ float value_of(float v)
{
    const float r = DT == MOE_BF16 ? __bfloat162float(__float2bfloat16_rn(v)) : __half2float(__float2half_rn(v));
    return fabsf(r) <= 3.4e38f ? r : 0.f;
}

__device__ __forceinline__ float field_value(uint32_t field) { return __uint_as_float(field << 23); }

// mma with nothing to add to
template <int DT>
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    static_assert(DT == MOE_F16, "");
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// eight 16-bit elements at row * K + k as they are; elements past K read 0
__device__ __forceinline__ uint4 load8_raw(const void *p, int64_t row, int K, int k, bool wide)
{
    const uint16_t *q = static_cast<const uint16_t *>(p) + row * K + k;
    if (wide)   // K is a multiple of 8
        return k < K ? __ldg(reinterpret_cast<const uint4 *>(q)) : make_uint4(0, 0, 0, 0);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t lo = k + 2 * j < K ? __ldg(q + 2 * j) : 0u, hi = k + 2 * j + 1 < K ? __ldg(q + 2 * j + 1) : 0u;
        w[j] = lo | hi << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight codes to eight float16 values, in order.  The conversion instruction does two at a time: 37
// words a nanosecond on an SM, where shifts and masks did 14 and a stream at full rate needs 12.
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t (&d)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(w));
}

// the four scales of w's bytes, exactly (0: 2^-127, 255: NaN)
__device__ __forceinline__ void scales_to_float(uint32_t w, float (&s)[4])
{
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %0, a;\n\tcvt.rn.bf16x2.ue8m0x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    s[0] = __uint_as_float(lo << 16);
    s[1] = __uint_as_float(lo & 0xffff0000u);
    s[2] = __uint_as_float(hi << 16);
    s[3] = __uint_as_float(hi & 0xffff0000u);
}

__device__ __forceinline__ uint32_t half2_mul(uint32_t a, __half2 b)
{
    const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&a), b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// ---------------------------------------------------------------- the grid-wide waits
//
// The launch is cooperative: all blocks run at once.  The workspace comes uninitialised, so the first
// wait goes by words that need no initial value: block b writes the call's tag (64 random-looking
// bits, different for each call) into its own, block 0 reads them all and then writes the tag into
// the word that the others read.  The later waits count arrivals in words that block 0 cleared before
// the first.  One thread a block reads one word: 152 blocks that each read 152 words held one another
// up for microseconds.  A launch replayed from a graph has the same tag each time, so a block never leaves
// without clearing its word (block 0 the common one): after the last wait, when all are through the first,
// or where it gives up, which can only make others give up too.  A wait that lasts p.wait_ns all the same
// gives up and returns false.
struct Waits {
    unsigned long long go, arrived[2];
    unsigned long long block[];
};

template <typename Done>
__device__ __forceinline__ bool poll(const Params &p, const unsigned long long *word, Done done)
{
    uint64_t t0 = 0;   // the timer is slow to read: not before a wait has become a long one
    for (uint32_t it = 1;; ++it) {
        unsigned long long v;
        asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(word) : "memory");
        if (done(v))
            return true;
        if (it % 256 == 0) {
            const uint64_t now = mrr::global_timer_ns();
            if (t0 == 0)
                t0 = now;
            else if (now - t0 > p.wait_ns)
                return false;
        }
    }
}

__device__ __forceinline__ void publish(unsigned long long *word, unsigned long long v)
{
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(word), "l"(v) : "memory");
}

// which: 0, or 1 and 2 for the counted ones
template <int kThreads>
__device__ __forceinline__ bool grid_wait(const Params &p, int which, int *s_ok)
{
    Waits *w = p.waits;
    const unsigned blocks = gridDim.x + (p.short_of && __ldcg(p.short_of) == 1u + which);
    auto is_tag = [&](unsigned long long v) { return v == p.tag; };
    bool ok = true;
    if (threadIdx.x == 0)
        *s_ok = 1;
    __syncthreads();
    if (which > 0) {
        if (threadIdx.x == 0) {
            asm volatile("red.release.gpu.global.add.u64 [%0], 1;" ::"l"(&w->arrived[which - 1]) : "memory");
            ok = poll(p, &w->arrived[which - 1], [&](unsigned long long v) { return v >= blocks; });
        }
    } else if (blockIdx.x > 0) {
        if (threadIdx.x == 0) {
            publish(&w->block[blockIdx.x], p.tag);
            ok = poll(p, &w->go, is_tag);
        }
    } else {
        for (int i = threadIdx.x; i < (int)blocks; i += kThreads)
            if (i > 0)
                ok = ok && poll(p, &w->block[i], is_tag);
        if (!ok)
            *s_ok = 0;
        __syncthreads();
        if (threadIdx.x == 0 && *s_ok)
            publish(&w->go, p.tag);
    }
    if (!ok)
        *s_ok = 0;
    __syncthreads();
    return *s_ok != 0;
}

// ---------------------------------------------------------------- routing of one token by one warp

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// order-preserving map of a score to a key above 0 (0 marks an expert out of the choice)
__device__ __forceinline__ uint32_t order_key(float f)
{
    const uint32_t b = __float_as_uint(f + 0.0f);
    return max(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u), 1u);
}

__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float(key ^ ((uint32_t)((int32_t)~key >> 31) | 0x80000000u));
}

// The `count` largest of n keys, ties to the lower index, by one warp: pick(i, index, key) is called
// by every lane.  A key taken is set to 0; the other keys are above 0 and at least `count`.
template <typename Pick>
__device__ __forceinline__ void pick_largest(uint32_t *key, int n, int count, Pick pick)
{
    const int lane = threadIdx.x % 32;
    uint32_t best = 0u;
    int at = lane;
    auto scan = [&]() {   // the best of this lane's
        best = 0u;
#pragma unroll 4
        for (int e = lane; e < n; e += 32)
            if (key[e] > best) {
                best = key[e];
                at = e;
            }
    };
    scan();
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
        const uint32_t top = __reduce_max_sync(kFull, best);
        const uint32_t e = __reduce_min_sync(kFull, best == top && best ? (uint32_t)at : 0xffffffffu);
        pick(i, (int)e, top);
        if ((int)(e % 32) == lane) {
            key[e] = 0u;
            scan();
        }
    }
    __syncwarp();
}

// The formulas of mrr_gating.h for one token by one warp: key holds its E logits (as float bits), with
// room for as many words behind them.  Whatever the logits hold, the k experts are different and in
// range.
static __device__ __noinline__ void route(const Params &p, uint32_t *key, const float *bias, uint16_t *expert, float *weight)
{
    const int lane = threadIdx.x % 32, E = p.E;
    float sum = 0.f;
    if (p.norm_type == 0) {
        float mx = -INFINITY;
        for (int e = lane; e < E; e += 32)
            mx = fmaxf(mx, __uint_as_float(key[e]));
        mx = key_value(__reduce_max_sync(kFull, order_key(mx)));
#pragma unroll 2
        for (int e = lane; e < E; e += 32) {
            const float v = expf(__uint_as_float(key[e]) - mx);
            key[e] = __float_as_uint(v);
            sum += v;
        }
        sum = warp_sum(sum);
    }
#pragma unroll 2
    for (int e = lane; e < E; e += 32) {
        float v = __uint_as_float(key[e]);
        if (p.norm_type == 0)
            v = v / sum;
        else if (p.norm_type == 1)
            v = 1.f / (1.f + expf(-v));
        else
            v = v > 20.f ? v + log1pf(expf(-v)) : log1pf(expf(v));
        key[e] = order_key(bias ? v + bias[e] : v);
    }
    __syncwarp();
    if (p.k_group < p.group_count) {
        uint32_t *group = key + E;
        const int size = E / p.group_count;
        for (int g = lane; g < p.group_count; g += 32) {
            uint32_t a = 0u, b = 0u;   // the two best of the group
            int e = lane % size;       // neighbouring lanes start at different banks
#pragma unroll 4
            for (int i = 0; i < size; ++i) {
                const uint32_t v = key[g * size + e];
                b = max(b, min(a, v));
                a = max(a, v);
                e = e + 1 == size ? 0 : e + 1;
            }
            group[g] = p.select_mode == 1 ? order_key(key_value(a) + key_value(b)) : a;
        }
        __syncwarp();
        pick_largest(group, p.group_count, p.k_group, [](int, int, uint32_t) {});
        for (int e = lane; e < E; e += 32)
            if (group[e / size])   // not picked
                key[e] = 0u;
        __syncwarp();
    }
    float total = 0.f;
    pick_largest(key, E, p.k, [&](int i, int e, uint32_t top) {
        const float v = key_value(top);
        total += v;
        if (lane == 0) {
            expert[i] = (uint16_t)e;
            weight[i] = v;
        }
    });
    for (int i = lane; i < p.k; i += 32)
        weight[i] = weight[i] / (total + p.eps) * p.rsf;
    __syncwarp();
}

// ---------------------------------------------------------------- one warp's weight stream

// Where a warp's stream of weight stages stands: first its units of this block's up items, then
// those of its down items.  A unit is one stage: 16 gate rows and their 16 up rows x 128 bytes, or 16
// rows x 256 bytes.
struct Cursor {
    int phase;                 // 0: up, 1: down, 2: over
    int item, expert, chunk;   // expert: index among the active ones; chunk: along K
    int part, last;            // down: the share of the expert's K that this warp is in; its end
    int row;                   // first weight row
    const uint8_t *scale_src;  // this lane's 8 scale bytes of chunk 0; null if there is no such row
};

// kSplit: y has few rows (H up to half of 16 a block), and several blocks share a down item: each writes its
// sums, and the last to come adds them up, always in the same order.  39 tokens, 248 experts of 556 x 1439 in
// float16 (35 items): 557 -> 304 us; 13 tokens, 12 experts of 153 x 1455: 50 -> 33; where items are not shared
// the code for it costs up to 5 %, so it is an instance of its own.
template <int DT, int WDT, int kRegime, bool kWide, bool kSplit>
struct Layer {
    static constexpr bool kMany = kRegime != kFew;            // more than 8 tokens
    static constexpr bool kMx = WDT == MOE_MXFP4;
    static constexpr int NT = tiles_for(kMx, kRegime);
    static constexpr int kWarps = warps_of(kMx, kWide, kRegime), kThreads = 32 * kWarps;
    static constexpr int kStages = stages_of(kMx, kWide, kRegime);
    static constexpr int MDT = kMx ? MOE_F16 : DT;            // the matrix instructions' type
    static constexpr bool kScaled = MDT == MOE_F16;           // h carries a power of two for each tile
    static constexpr int kPitch = pitch_of(kWide), kSlab = 16 * kPitch, kStage = stage_of(kWide);
    static constexpr int kSlabK = kMx ? 256 : 64;             // elements of K in 128 bytes
    static constexpr int kUpK = kSlabK, kDownK = 2 * kSlabK;  // and in a stage

    const Params &p;
    uint8_t *smem;
    int warp, lane, g, t;
    int row;                     // of a slab's rows 0 .. 7, the one this lane's operands come from
    int lane_at;                 // where in a slab they are
    uint32_t bars;               // this warp's barriers, one a stage
    bool dead;                   // a wait has given up: results do not matter any more
    uint32_t held[2];            // scale bytes on their way through registers, for stage held_slot (-1: none)
    int held_slot;
    int nact, up_items, up_units, up_tiles, down_items, down_chunks, down_parts;
    bool solo;                   // up items are single warps', not the block's
    int splits_, split_, down_first_;   // kSplit: blocks of a down item; which of them this is; its first item
    int up_first, up_stride, up_begin, up_step;   // this warp's items, and its units of one
    const uint16_t *act, *start, *cols;
    const uint8_t *tokens;       // of the columns (kMany)

    __device__ Layer(const Params &p_, uint8_t *sm) : p(p_), smem(sm)
    {
        warp = threadIdx.x / 32;
        lane = threadIdx.x % 32;
        g = lane / 4;
        t = lane % 4;
        // The copies' swizzle puts 16-byte piece c of row r at c ^ (r % 8).  16-bit weights: lanes g and
        // g + 1 of a 128-byte read take rows 4 apart, and so the two halves of the banks.
        row = g >> 1 | (g & 1) << 2;
        if (kWide)
            lane_at = kMx ? row * 128 + row * 16 + 4 * t : row * 128 + ((t ^ row) << 4);
        else
            lane_at = row * kPitch + t * (kMx ? 4 : 16);
        bars = mrr::smem_addr(sm + p.sm_bar) + warp * kStages * 8;
        dead = false;
        held_slot = -1;
        act = reinterpret_cast<const uint16_t *>(sm + p.sm_act);
        start = reinterpret_cast<const uint16_t *>(sm + p.sm_start);
        cols = reinterpret_cast<const uint16_t *>(sm + p.sm_cols);
        tokens = sm + p.sm_tokens;
        if (threadIdx.x < kWarps * kStages)   // the tiled copies, or every lane's, and (scales) every lane's
            mrr::mbar_init(mrr::smem_addr(sm + p.sm_bar) + threadIdx.x * 8,
                           (kWide ? 1 : 32) + (kMx ? 32 : 0) + (p.short_of && __ldcg(p.short_of) == kShortStages));
        mrr::mbar_init_fence();
    }

    __device__ __forceinline__ uint8_t *stage(int slot) const { return smem + (warp * kStages + slot) * kStage; }
    __device__ __forceinline__ uint8_t *scales(int slot) const
    {
        return smem + p.sm_scales + (warp * kStages + slot) * kStageScales;
    }

    __device__ void sizes(int active)
    {
        nact = active;
        up_tiles = (p.I + 15) / 16;
        up_items = nact * up_tiles;
        up_units = (p.H + kUpK - 1) / kUpK;
        // An up item is worked off by the block, its warps splitting K and joining their sums, or by one warp,
        // which needs no join.  Which takes less, in units of a stage's time: the block's share of K and
        // about one for each join, times its items; or all of K, a fifth more for the more scattered
        // reads of the weights, times the warp's items.  48 tokens, 64 experts of 7168 x 2048 in bfloat16:
        // the block 926 us, warps 1000; 39 tokens, 248 experts of 556 x 1439 in float16: 477 and 300; 32
        // tokens, 64 MXFP4 experts of 7168 x 2048: 413 and 350; 2 tokens, 18 experts of 5015 x 196: 46 and 88.
        const int blocks = gridDim.x, joins = !kMany ? 1 : min(NT, (p.T * p.k + 8 * nact - 1) / (8 * nact));
        const int joint = (up_items + blocks - 1) / blocks * ((up_units + kWarps - 1) / kWarps + joins);
        const int alone = (up_items + kWarps * blocks - 1) / (kWarps * blocks) * up_units;
        solo = 5 * (int64_t)joint > 6 * (int64_t)alone;
        up_first = blockIdx.x + (solo ? warp * blocks : 0);
        up_stride = solo ? kWarps * blocks : blocks;
        up_begin = solo ? 0 : warp;
        up_step = solo ? 1 : kWarps;
        down_items = (p.H + 15) / 16;
        down_chunks = (p.I + kDownK - 1) / kDownK;
        if (kSplit) {
            splits_ = max(1, min(min(blocks / down_items, kMaxSplits), nact * down_chunks / (2 * kWarps)));
            split_ = splits_ > 1 ? blockIdx.x / down_items : 0;
            down_first_ = splits_ == 1 ? blockIdx.x : split_ < splits_ ? blockIdx.x - split_ * down_items : down_items;
        }
        // an expert's K is cut into shares, taken by the warps in turn: single chunks, or (where a
        // change of expert costs something) as few as give every warp four or more
        down_parts = !kMany ? down_chunks : min(down_chunks, (4 * down_stride() + nact - 1) / nact);
    }

    __device__ __forceinline__ int splits() const { return kSplit ? splits_ : 1; }
    __device__ __forceinline__ int split() const { return kSplit ? split_ : 0; }
    __device__ __forceinline__ int down_first() const { return kSplit ? down_first_ : (int)blockIdx.x; }
    __device__ __forceinline__ int down_stride() const { return splits() * kWarps; }

    // point the cursor at the rows of its item and expert
    __device__ __forceinline__ void aim(Cursor &c) const
    {
        const int r = lane % 16;
        if (c.phase == 0) {
            const int i0 = (c.item - c.expert * up_tiles) * 16;
            c.row = act[c.expert] * 2 * p.I + i0;
            if (kMx)
                c.scale_src = i0 + r < p.I ? p.w13_s + (int64_t)(c.row + r + lane / 16 * p.I) * scale_row_bytes(p.H) : nullptr;
        } else if (c.phase == 1) {
            const int n0 = c.item * 16;
            c.row = act[c.expert] * p.H + n0;
            if (kMx)
                c.scale_src = n0 + r < p.H ? p.w2_s + (int64_t)(c.row + r) * scale_row_bytes(p.I) + lane / 16 * 8 : nullptr;
        }
    }

    // the chunk after c's in the down product, within its item; false if there is none
    __device__ __forceinline__ bool next_chunk(Cursor &c) const
    {
        if (++c.chunk < c.last)
            return true;
        c.part += down_stride();
        return enter_part(c);
    }

    __device__ __forceinline__ bool first_chunk(Cursor &c) const
    {
        c.part = split() * kWarps + warp;
        c.expert = 0;
        return enter_part(c);
    }

    __device__ __forceinline__ bool enter_part(Cursor &c) const
    {
        while (c.part >= down_parts) {
            c.part -= down_parts;
            if (++c.expert >= nact)
                return false;
        }
        c.chunk = !kMany ? c.part : c.part * down_chunks / down_parts;
        c.last = !kMany ? c.part + 1 : (c.part + 1) * down_chunks / down_parts;
        return true;
    }

    __device__ __forceinline__ Cursor first_unit() const
    {
        Cursor c;
        c.phase = 0;
        c.item = up_first;
        c.chunk = up_begin;
        if (c.item >= up_items || up_begin >= up_units)
            first_down(c);
        else
            c.expert = c.item / up_tiles;
        aim(c);
        return c;
    }

    __device__ __forceinline__ void first_down(Cursor &c) const
    {
        c.item = down_first();
        c.phase = c.item < down_items && first_chunk(c) ? 1 : 2;
    }

    __device__ __forceinline__ void advance(Cursor &c) const
    {
        if (c.phase == 0) {
            c.chunk += up_step;
            if (c.chunk < up_units)
                return;
            c.chunk = up_begin;
            c.item += up_stride;
            if (c.item >= up_items)
                first_down(c);
            else
                c.expert = c.item / up_tiles;
        } else {
            const int e = c.expert;
            if (next_chunk(c)) {
                if (c.expert == e)
                    return;
            } else {
                c.item += gridDim.x;
                c.phase = c.item < down_items && first_chunk(c) ? 1 : 2;
            }
        }
        aim(c);
    }

    // start bringing the cursor's unit into stage `slot`: slab 0 holds the gate rows or the chunk's first
    // 128 bytes, slab 1 the up rows or the other 128 bytes
    template <bool kUp>
    __device__ __forceinline__ void fill(int slot, const Cursor &c)
    {
        const uint32_t to = mrr::smem_addr(stage(slot)), bar = bars + 8 * slot;
        if (kWide) {
            if (lane == 0) {
                mrr::mbar_arrive_expect_tx(bar, 2 * kSlab);
                const CUtensorMap *map = kUp ? &p.w13_map : &p.w2_map;
                tc::load_box(to, map, c.chunk * (kUp ? 128 : 256), c.row, bar);
                tc::load_box(to + kSlab, map, c.chunk * (kUp ? 128 : 256) + (kUp ? 0 : 128), c.row + (kUp ? p.I : 0), bar);
            }
        } else {
            // Rows that begin at any byte: the nine aligned 16-byte pieces that hold 128 bytes of each, cut off
            // at the row's end.  Lanes take 8 pieces of 4 rows at a time, the ninth of all 32 rows last.  Bound by
            // the instructions of copies and shifts: 7 tokens, 60 experts of 2055 x 1399 in float16 take
            // 151 us (2056 x 1400: 104); by 33 aligned words a row it was 197, by loads of single elements 655.
            const int K = kUp ? p.H : p.I;
            const int64_t bytes = kMx ? K / 2 : 2 * (int64_t)K;
            const uintptr_t all = reinterpret_cast<uintptr_t>(kUp ? p.w13 : p.w2);
            const int n = (kUp ? p.I : p.H) - (kUp ? (c.item - c.expert * up_tiles) * 16 : c.item * 16);
            const int64_t first = (int64_t)c.chunk * (kUp ? 128 : 256);
            const uintptr_t at = all + (int64_t)c.row * bytes + first;   // slab 0's first row
            const uintptr_t at1 = at + (kUp ? p.I * bytes : 128);        // slab 1's
            if ((at & ~(uintptr_t)15) < all) {
                // the tensor's first piece holds bytes that are not the tensor's: byte by byte
#pragma unroll 1
                for (int i = lane; i < 32 * kPitch / 4; i += 32) {
                    const int r = i / (kPitch / 4) % 16;
                    const uintptr_t row_at = (i / (kPitch / 4) < 16 ? at : at1) + r * bytes;
                    const uintptr_t from = (row_at & ~(uintptr_t)15) + i % (kPitch / 4) * 4;
                    const uintptr_t end = row_at - first - (!kUp && i / (kPitch / 4) >= 16 ? 128 : 0) + bytes;
                    uint32_t v = 0u;
                    for (int b = 0; b < 4; ++b)
                        if (r < n && from + b >= all && from + b < end)
                            v |= (uint32_t)__ldg(reinterpret_cast<const uint8_t *>(from + b)) << (8 * b);
                    reinterpret_cast<uint32_t *>(stage(slot))[i] = v;
                }
            } else {
                const bool whole = n >= 16 && first + (kUp ? 128 : 256) <= bytes;   // nothing to cut off
#pragma unroll
                for (int slab = 0; slab < 2; ++slab) {
                    const uintptr_t slab_at = (slab ? at1 : at) & ~(uintptr_t)15;
                    uint32_t off = (uint32_t)((slab ? at1 : at) & 15) + lane / 8 * (uint32_t)bytes;   // of the lane's row
                    const uint32_t dst = to + slab * kSlab + lane / 8 * kPitch + lane % 8 * 16;
                    const uintptr_t from = slab_at + lane % 8 * 16;
                    if (whole) {
#pragma unroll
                        for (int r = 0; r < 16; r += 4, off += 4 * (uint32_t)bytes)
                            copy16(dst + r * kPitch, from + (off & ~15u));
                    } else {
                        const int left = (int)(bytes - first) - (!kUp && slab ? 128 : 0) - lane % 8 * 16;
#pragma unroll
                        for (int r = 0; r < 16; r += 4, off += 4 * (uint32_t)bytes) {
                            const int some = r + lane / 8 < n ? min(max(left + (int)(off & 15u), 0), 16) : 0;
                            copy16(dst + r * kPitch, some ? from + (off & ~15u) : reinterpret_cast<uintptr_t>(p.status), some);
                        }
                    }
                }
                const int r = lane % 16;
                const uintptr_t row_at = (lane < 16 ? at : at1) + r * bytes, from = (row_at & ~(uintptr_t)15) + 128;
                const int64_t left = (int64_t)(row_at - from) - first - (!kUp && lane >= 16 ? 128 : 0) + bytes;
                const int some = r < n ? (int)max((int64_t)0, min((int64_t)16, left)) : 0;
                copy16(to + lane * kPitch + 128, some ? from : reinterpret_cast<uintptr_t>(p.status), some);
            }
            copies_arrive(bar);
        }
        if (kMx) {
            // 8 scale bytes a lane: [slab][row].  Bytes that stand for no block, the unused one of a last pair
            // among them, read 0: 2^-127 leaves the zeros past K what they are, where a 255 would make them NaN.
            const int at = c.chunk * (kUp ? 8 : 16), left = ((kUp ? p.H : p.I) + kBlock - 1) / kBlock - at - (kUp ? 0 : lane / 16 * 8);
            const bool ok = c.scale_src && left > 0;
            if (kUp ? p.s13_wide : p.s2_wide) {
                // the address counts even where nothing is read: one that is aligned whatever the scales' are
                copy8(mrr::smem_addr(scales(slot)) + lane * 8,
                      ok ? c.scale_src + at : reinterpret_cast<const uint8_t *>(p.status), ok ? min(left, 8) : 0);
                copies_arrive(bar);
            } else {   // two bytes at a time, put into the stage at the next issue: they have come by then
                held[0] = held[1] = 0u;
                held_slot = slot;
                if (ok)
#pragma unroll
                    for (int b = 0; b < 8; b += 2)
                        if (b < left)
                            held[b / 4] |= load_pair(c.scale_src + at + b, b + 1 < left) << (8 * (b % 4));
            }
        }
    }

    // two bytes at any address, or one
    __device__ __forceinline__ uint32_t load_pair(const uint8_t *p_, bool both) const
    {
        if (both && reinterpret_cast<uintptr_t>(p_) % 2 == 0)
            return __ldg(reinterpret_cast<const uint16_t *>(p_));
        return (uint32_t)__ldg(p_) | (both ? (uint32_t)__ldg(p_ + 1) << 8 : 0u);
    }

    __device__ __forceinline__ void put_held()
    {
        if (kMx && held_slot >= 0) {
            *reinterpret_cast<uint2 *>(scales(held_slot) + lane * 8) = make_uint2(held[0], held[1]);
            tc::mbar_arrive(bars + 8 * held_slot);
            held_slot = -1;
        }
    }

    __device__ __forceinline__ void issue(Cursor &c, int slot)
    {
        put_held();
        if (c.phase == 0)
            fill<true>(slot, c);
        else if (c.phase == 1)
            fill<false>(slot, c);
        if (c.phase < 2)
            advance(c);
    }

    // the stage's copies have landed, or the warp has given up, and brings no more: `next` is over
    __device__ __forceinline__ void landed(int slot, uint32_t parity, Cursor &next)
    {
        if (!dead) {
            uint64_t t0 = 0;   // the timer is slow to read: not before a wait has become a long one
            for (uint32_t it = 1; !mrr::mbar_try_wait(bars + 8 * slot, parity); ++it)
                if (it % 1024 == 0) {
                    const uint64_t now = mrr::global_timer_ns();
                    if (t0 == 0)
                        t0 = now;
                    else if (now - t0 > p.wait_ns) {
                        dead = true;
                        break;
                    }
                }
            dead = __any_sync(kFull, dead);
            if (dead)
                next.phase = 2;
        }
        __syncwarp();
    }

    // A warp that has given up leaves no copy in flight: each stage's have a moment to land.  At most one of a
    // barrier's two phases is not over.
    __device__ __forceinline__ void settle() const
    {
        for (int s = 0; s < kStages; ++s)
            for (int b = 0; b < 2; ++b)
                mrr::mbar_wait_bounded(bars + 8 * s, b, 1000000ull);
        asm volatile("cp.async.wait_all;" ::: "memory");
    }

    // Narrow rows: by how many bytes what this lane reads of the unit's slabs (rows `row` and `row` + 8, and
    // the same of the up rows) lies past an aligned piece.
    uint32_t shift[2][2];

    __device__ __forceinline__ void place_rows(const void *w, int row0, int K, int second)
    {
        if (kWide)
            return;
        const uint32_t bytes = kMx ? K / 2 : 2 * K, base = (uint32_t)reinterpret_cast<uintptr_t>(w);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                shift[m][r] = (base + (uint32_t)(row0 + row + 8 * r + m * second) * bytes) & 15u;
    }

    // the 16 bytes from byte d of two pieces
    __device__ __forceinline__ uint4 shifted(const uint4 &lo, const uint4 &hi, uint32_t d) const
    {
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        uint32_t x[6], y[5];
#pragma unroll
        for (int i = 0; i < 6; ++i)
            x[i] = d & 8u ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i)
            y[i] = d & 4u ? x[i + 1] : x[i];
        const uint32_t bits = d % 4u * 8u;
        return make_uint4(__funnelshift_r(y[0], y[1], bits), __funnelshift_r(y[1], y[2], bits),
                          __funnelshift_r(y[2], y[3], bits), __funnelshift_r(y[3], y[4], bits));
    }

    // Token operands of one step (a stage, or half of one), kGroups groups of 32 k, for kCols column tiles: this lane's 8 elements
    // of each.  Every register is loaded with the next step's value as soon as it has been used, so
    // that a step's time hides the loads.
    static constexpr int kCols = kRegime == kDense || NT == 1 ? NT : 2;
    static constexpr int kSlabGroups = kSlabK / 32, kUpGroups = kUpK / 32;
    // Parts of h that more than 4 tokens' columns take one after the other.  One float16 part is enough
    // where y is bfloat16: it adds 2^-12 to an error of 2^-9.
    static constexpr int kParts = kMx && DT == MOE_BF16 ? 1 : 2;
    static constexpr int kStored = kMany ? kParts : 2;   // in memory
    // Down stages are worked off in steps, so that a step's operands fit the registers: MXFP4's are 16 groups long
    static __host__ __device__ constexpr int down_steps(int parts) { return kMx ? 2 * parts : kRegime == kDense ? parts : 1; }
    static __host__ __device__ constexpr int down_groups(int parts) { return kDownK / 32 / down_steps(parts); }
    template <int kGroups, int kOf = 1>   // kOf: parts
    struct Tokens {
        uint4 v[kOf][kCols][kGroups];
        uint32_t tile[kCols][kGroups];   // exponents of the tiles' powers of two (h in float16)
    };
    // Where a column's operands come from, this lane's part: null pointers for a column that is not there.
    struct Column {
        const uint16_t *v = nullptr;
        const uint8_t *tile = nullptr;
        uint32_t field = 127u;           // exponent of the power of two that the token's sums carry
    };

    template <bool kUp, int kGroups, int kOf>
    __device__ __forceinline__ void load(Tokens<kGroups, kOf> &b, int j, int i, const Column &c, int k0) const
    {
        const uint16_t *from = c.v + (kUp ? 1 : kStored) * (k0 + 32 * i);
        uint4 v = make_uint4(0, 0, 0, 0), w = v;
        if (c.v) {
            if constexpr (kOf == 2)   // both parts, 32 bytes
                asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w), "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                             : "l"(from));
            else
                v = *reinterpret_cast<const uint4 *>(from);
        }
        b.v[0][j][i] = v;
        if constexpr (kOf == 2)
            b.v[1][j][i] = w;
        if (!kUp && kScaled) {
            uint32_t f = 253u;
            if (c.v)
                f = c.tile[k0 / 16 + 2 * i];
            b.tile[j][i] = f;
        }
    }

    template <bool kUp, int kGroups, int kOf>
    __device__ __forceinline__ void load_all(Tokens<kGroups, kOf> &b, const Column (&c)[kCols], int k0) const
    {
#pragma unroll
        for (int j = 0; j < kCols; ++j)
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
                load<kUp>(b, j, i, c[j], k0);
    }

    // The products of a step: two row tiles, one a slab (kUp), or one whose K runs on from slab to slab,
    // from the stage's group g0, against column tiles j0 .. j0 + kN - 1.  kNext: their operands are b, which is
    // loaded anew from `next` at k1; else they are loaded here from `now` at k1, four groups at a time.
    // Past K both operands are zeros.
    template <bool kUp, int kN, bool kNext, int kGroups, int kHeld, int kOf>
    __device__ __forceinline__ void multiply(int slot, int g0, int j0, Tokens<kHeld, kOf> &b, const Column (&now)[kCols],
                                             const Column (&next)[kCols], int k1, float (&acc)[2][NT][4]) const
    {
        constexpr int kTiles = kUp ? 2 : 1, kBatch = kHeld < kGroups ? kHeld : kGroups;
        const int stage_at = (warp * kStages + slot) * kStage + lane_at;   // kWide: a multiple of 1024, and lane_at
        uint2 sc[2][2];   // 8 scale bytes of rows `row` and `row` + 8
        if constexpr (kMx)
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    sc[m][r] = *reinterpret_cast<const uint2 *>(scales(slot) + (kUp ? m : g0 / kSlabGroups) * 128 + r * 64 + row * 8);
        float s[2][2][4];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int q = (g0 + i) % kSlabGroups, slab = kUp ? 0 : (g0 + i) / kSlabGroups;
            const uint8_t *from = kWide ? smem + (stage_at ^ (kMx ? q << 4 : q << 6)) + slab * kSlab
                                        : smem + stage_at + (kMx ? q << 4 : q << 6) + slab * kSlab;
            if (!kNext && i % kBatch == 0)
#pragma unroll
                for (int j = 0; j < kN; ++j)
#pragma unroll
                    for (int h = 0; h < kBatch; ++h)
                        load<kUp>(b, j, h, now[j], k1 + 32 * i);
            uint32_t a[kTiles][2][4];
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r) {   // slab rows `row` and `row` + 8
                    const uint8_t *piece = from + m * kSlab + r * 8 * kPitch;
                    if constexpr (kMx) {
                        uint32_t w;
                        if (kWide) {
                            w = *reinterpret_cast<const uint32_t *>(piece);
                        } else {
                            const uint32_t *words = reinterpret_cast<const uint32_t *>(piece + (shift[m][r] & 12u));
                            w = __funnelshift_r(words[0], words[1], shift[m][r] % 4u * 8u);
                        }
                        codes_to_half(w, a[m][r]);
                        if (i % 4 == 0)
                            scales_to_float(q < 4 ? sc[m][r].x : sc[m][r].y, s[m][r]);
                    } else {
                        uint4 v = *reinterpret_cast<const uint4 *>(piece);
                        if (!kWide)
                            v = shifted(v, *reinterpret_cast<const uint4 *>(piece + 16), shift[m][r]);
                        a[m][r][0] = v.x, a[m][r][1] = v.y, a[m][r][2] = v.z, a[m][r][3] = v.w;
                    }
                }
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const int at = kNext ? i : i % kBatch;
                __half2 f;   // the token's power of two over the tile's: at most 1
                if (!kUp && kScaled)
                    f = __float2half2_rn(field_value(127u - min(b.tile[j][at] - now[j].field, 126u)));
#pragma unroll
                for (int part = 0; part < kOf; ++part) {
                    uint4 x = b.v[part][j][at];
                    if (!kUp && kScaled)
                        x = make_uint4(half2_mul(x.x, f), half2_mul(x.y, f), half2_mul(x.z, f), half2_mul(x.w, f));
#pragma unroll
                    for (int m = 0; m < kTiles; ++m) {
                        // one row tile: two chains of sums, the parts' or so that an instruction waits for the last but one
                        float(&to)[4] = acc[kUp ? m : kOf == 2 ? part : i % 2][j0 + j];
                        if constexpr (kMx) {
                            float d[4];
                            mma_first<MDT>(d, a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1], x.x, x.y);
                            mma<MDT>(d, a[m][0][2], a[m][1][2], a[m][0][3], a[m][1][3], x.z, x.w);
                            to[0] = fmaf(s[m][0][i % 4], d[0], to[0]);
                            to[1] = fmaf(s[m][0][i % 4], d[1], to[1]);
                            to[2] = fmaf(s[m][1][i % 4], d[2], to[2]);
                            to[3] = fmaf(s[m][1][i % 4], d[3], to[3]);
                        } else {
                            mma<MDT>(to, a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1], x.x, x.y);
                            mma<MDT>(to, a[m][0][2], a[m][1][2], a[m][0][3], a[m][1][3], x.z, x.w);
                        }
                    }
                }
            }
            if (kNext)
#pragma unroll
                for (int j = 0; j < kCols; ++j)
                    load<kUp>(b, j, i, next[j], k1);
        }
    }

    // All nt column tiles of a step: the first kCols, whose operands are b, and (rarely) more, whose
    // operands are loaded here from column(tile) at k0.
    template <bool kUp, int kGroups, int kOf, typename Of>
    __device__ __forceinline__ void multiply_all(int slot, int g0, int nt, Tokens<kGroups, kOf> &b,
                                                 const Column (&now)[kCols], const Column (&next)[kCols], int k0, int k1,
                                                 float (&acc)[2][NT][4], Of column) const
    {
        if (kCols == 1 || nt == 1)
            multiply<kUp, 1, true, kGroups>(slot, g0, 0, b, now, next, k1, acc);
        else if (kCols > 2 && nt == 2)
            multiply<kUp, 2, true, kGroups>(slot, g0, 0, b, now, next, k1, acc);
        else
            multiply<kUp, kCols, true, kGroups>(slot, g0, 0, b, now, next, k1, acc);
#pragma unroll
        for (int j = kCols; j < NT; j += kCols) {
            if (j >= nt)
                break;
            Column more[kCols];
            for (int c = 0; c < kCols; ++c)
                if (j + c < nt)
                    more[c] = column(j + c);
            Tokens<kGroups < 4 / kOf ? kGroups : 4 / kOf, kOf> x;
            multiply<kUp, kCols, false, kGroups>(slot, g0, j, x, more, more, k0, acc);
        }
    }

    // token of column c of active expert ai, which exists
    __device__ __forceinline__ int token_of(int ai, int c) const { return !kMany ? c : (int)tokens[start[ai] + c]; }

    // assignment of column c of active expert ai, or -1.  Up to 8 tokens: column = token.
    __device__ __forceinline__ int column_of(int ai, int c) const
    {
        if (!kMany) {
            const uint16_t a = cols[ai * 8 + c];
            return a == 0xffffu ? -1 : (int)a;
        }
        const int s = start[ai];
        return c < (int)start[ai + 1] - s ? (int)cols[s + c] : -1;
    }

    __device__ __forceinline__ int tiles_of(int ai) const
    {
        return !kMany ? 1 : ((int)start[ai + 1] - (int)start[ai] + 7) / 8;
    }

    // column c (of this lane) of active expert ai: its row of x, and of h
    __device__ __forceinline__ Column x_column(int ai, int tile) const
    {
        Column c;
        if (column_of(ai, 8 * tile + g) >= 0)
            c.v = p.xh + (int64_t)token_of(ai, 8 * tile + g) * p.Hp + 8 * t;
        return c;
    }

    __device__ __forceinline__ Column h_column(int ai, int tile) const
    {
        Column c;
        const int a = column_of(ai, 8 * tile + g);
        if (a >= 0) {
            c.v = p.h + kStored * ((int64_t)a * p.Ip + 8 * t);
            c.tile = p.h_field + (int64_t)a * (p.Ip / 16) + t / 2;
            c.field = field_of(token_of(ai, 8 * tile + g));
        }
        return c;
    }

    // the exponent of the power of two that token tok's down sums carry (float16)
    __device__ __forceinline__ uint32_t field_of(int tok) const
    {
        return kScaled ? f16_scale_field(__ldcg(p.h_max + tok)) : 127u;
    }

    __device__ __forceinline__ float *red(int buf) const
    {
        return reinterpret_cast<float *>(smem + p.sm_red) + buf * (kWarps * 256);
    }

    // this warp's 16 x 8 partial sums into red[.][warp][tile][row][column]
    __device__ __forceinline__ void put(float *r, int tile, const float (&d)[4], int row_) const
    {
        float *at = r + (warp * 2 + tile) * 128 + row_ * 8 + 2 * t;
        *reinterpret_cast<float2 *>(at) = make_float2(d[0], d[1]);
        *reinterpret_cast<float2 *>(at + 64) = make_float2(d[2], d[3]);
    }

    __device__ __forceinline__ float gather(const float *r, int tile, int row, int col) const
    {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            v += r[(w * 2 + tile) * 128 + row * 8 + col];
        return v;
    }

    // element i of assignment a's h
    __device__ __forceinline__ void store_h(int64_t a, int i, float v) const
    {
        const int64_t to = kStored * (a * p.Ip + i / 8 * 8) + i % 8;
        store1<MDT>(p.h, to, v);
        if (kStored == 2)
            store1<MDT>(p.h, to + 8, v - value_of<MDT>(v));
    }

    // h of column c of active expert ai, rows i0 + row and i0 + row + 8, from their gate and up sums: the
    // eight lanes that share t hold a column's 16 rows
    __device__ __forceinline__ void finish(const float *weight, int ai, int i0, int c, float g0, float g1, float u0, float u1) const
    {
        const int a = column_of(ai, c);
        float h[2] = {0.f, 0.f};
        int tok = 0;
        if (a >= 0) {
            tok = token_of(ai, c);
            const float s = kMx ? p.x_scale[tok] : 1.f, w = !kMany ? weight[a] : __ldcg(p.route_weight + a);
            const float gate[2] = {g0 * s, g1 * s}, upv[2] = {u0 * s, u1 * s};
#pragma unroll
            for (int b = 0; b < 2; ++b)   // rows past I: what the copy brought there is another row's
                h[b] = i0 + row + 8 * b < p.I ? gate[b] / (1.f + expf(-gate[b])) * upv[b] * w : 0.f;
        }
        if (kScaled) {
            uint32_t m = max(__float_as_uint(h[0]) & 0x7fffffffu, __float_as_uint(h[1]) & 0x7fffffffu);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
                m = max(m, __shfl_xor_sync(kFull, m, o));
            const uint32_t field = f16_scale_field(m);
            h[0] *= field_value(field), h[1] *= field_value(field);
            if (a >= 0 && g == 0) {
                p.h_field[(int64_t)a * (p.Ip / 16) + i0 / 16] = (uint8_t)field;
                atomicMax(p.h_max + tok, m);
            }
        }
        if (a >= 0) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
                store_h(a, i0 + row + 8 * b, h[b]);
        }
    }

    // The sum of two chains of one part, or of the parts'.  A first parts' sum that is not finite is all said: an
    // infinite weight times a second part, which may be 0 or of the other sign, would make it NaN.
    template <int kOf>
    static __device__ __forceinline__ float joined(float a, float b)
    {
        return kOf == 1 || fabsf(a) <= 3.4e38f ? a + b : a;
    }

    // this block's sum for row r of down item `item`, which exists
    __device__ __forceinline__ void give(int item, int tok, int r, float v) const
    {
        if (splits() == 1)
            store1<DT>(p.y, (int64_t)tok * p.H + item * 16 + r, v * field_value(254u - field_of(tok)));
        else
            __stcg(p.split + (((int64_t)split() * down_items + item) * p.T + tok) * 16 + r, v);
    }

    // the last of the item's blocks adds up what all have given
    __device__ __forceinline__ void add_shares(int item, int *last) const
    {
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
            *last = atomicAdd(p.split_count + item, 1u) == (unsigned)splits() - 1u;
            __threadfence();
        }
        __syncthreads();
        if (*last == 0)
            return;
        for (int i = threadIdx.x; i < 16 * p.T; i += kThreads) {
            const int r = i % 16, tok = i / 16;
            if (item * 16 + r >= p.H)
                continue;
            float v = 0.f;
#pragma unroll 4
            for (int q = 0; q < splits(); ++q)
                v += __ldcg(p.split + (((int64_t)q * down_items + item) * p.T + tok) * 16 + r);
            store1<DT>(p.y, (int64_t)tok * p.H + item * 16 + r, v * field_value(254u - field_of(tok)));
        }
    }

    // ------------------------------------------------------------ before the first wait

    // x's row t as the products take it: 16-bit, zeros past H, scaled (kMx); and the ends of its h rows
    __device__ void prepare_row(int tok)
    {
        uint32_t *s_max = reinterpret_cast<uint32_t *>(smem + p.sm_red);
        float scale = 1.f;
        if (kMx) {
            if (threadIdx.x == 0)
                *s_max = 0u;
            __syncthreads();
            uint32_t m = 0u;
            for (int i = threadIdx.x; i < p.H; i += kThreads)
                m = max(m, __float_as_uint(load1<DT>(p.x, (int64_t)tok * p.H + i)) & 0x7fffffffu);
            m = __reduce_max_sync(kFull, m);
            if (lane == 0)
                atomicMax(s_max, m);
            __syncthreads();
            const uint32_t field = f16_scale_field(*s_max);
            scale = field_value(field);
            if (threadIdx.x == 0)
                p.x_scale[tok] = field_value(254u - field);
            __syncthreads();
        } else if (threadIdx.x == 0) {
            p.x_scale[tok] = 1.f;
        }
        if (threadIdx.x == 0)
            p.h_max[tok] = 0u;
        const int end = (p.I + 15) / 16 * 16, pad = p.Ip - end;
        for (int i = threadIdx.x; i < p.k * pad; i += kThreads) {
            const int64_t a = (int64_t)tok * p.k + i / pad;
            store_h(a, end + i % pad, 0.f);
            if (i % pad % 16 == 0)
                p.h_field[a * (p.Ip / 16) + (end + i % pad) / 16] = 253;
        }
        for (int c = threadIdx.x; c < p.Hp / 8; c += kThreads) {
            uint4 v = load8_raw(p.x, tok, p.H, 8 * c, p.x_wide);
            if (kMx) {
                const float2 a = unpack2<DT>(v.x), b = unpack2<DT>(v.y), d = unpack2<DT>(v.z), e = unpack2<DT>(v.w);
                v = make_uint4(pack2<MDT>(a.x * scale, a.y * scale), pack2<MDT>(b.x * scale, b.y * scale),
                               pack2<MDT>(d.x * scale, d.y * scale), pack2<MDT>(e.x * scale, e.y * scale));
            }
            reinterpret_cast<uint4 *>(p.xh + (int64_t)tok * p.Hp)[c] = v;
        }
    }

    // partial logits of 16 experts over one of kparts shares of H, straight from global memory
    __device__ void router_item(int item)
    {
        const int et = item / p.kparts, part = item - et * p.kparts, chunks = (p.H + 127) / 128;
        const int lo = (int)((int64_t)chunks * part / p.kparts), hi = (int)((int64_t)chunks * (part + 1) / p.kparts);
        const int e0 = et * 16;
        constexpr int kTokenTiles = !kMany ? 1 : MOE_LAYER_MAX_TOKENS / 8;
        float acc[kTokenTiles][4] = {};
        for (int c = lo + warp; c < hi; c += kWarps) {
            uint4 a[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    a[r][q] = e0 + 8 * r + g < p.E ? load8_raw(p.wr, e0 + 8 * r + g, p.H, c * 128 + 32 * q + 8 * t, p.wr_wide)
                                                   : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < kTokenTiles; ++j) {
                if (8 * j >= p.T)
                    break;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 b = 8 * j + g < p.T ? load8_raw(p.x, 8 * j + g, p.H, c * 128 + 32 * q + 8 * t, p.x_wide)
                                                    : make_uint4(0, 0, 0, 0);
                    mma<DT>(acc[j], a[0][q].x, a[1][q].x, a[0][q].y, a[1][q].y, b.x, b.y);
                    mma<DT>(acc[j], a[0][q].z, a[1][q].z, a[0][q].w, a[1][q].w, b.z, b.w);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kTokenTiles; ++j) {
            if (8 * j >= p.T)
                break;
            put(red(j % 2), 0, acc[j], g);
            __syncthreads();
            if (threadIdx.x < 128) {
                const int row = threadIdx.x % 16, col = threadIdx.x / 16, tok = 8 * j + col;
                if (tok < p.T && e0 + row < p.E)
                    p.part[((int64_t)part * p.T + tok) * p.E + e0 + row] = gather(red(j % 2), 0, row, col);
            }
        }
        __syncthreads();
    }

    // ------------------------------------------------------------ between the waits: who goes where

    // the sums of the logits' parts for tokens tok .. tok + n - 1, into key (2 E words a token), and
    // the bias behind them, by the whole block
    __device__ void logits(int tok, int n, uint32_t *key, float *bias)
    {
        const int64_t plane = (int64_t)p.T * p.E;
        if (p.bias)
            for (int e = threadIdx.x; e < p.E; e += kThreads)
                bias[e] = load1<DT>(p.bias, e);
#pragma unroll 1
        for (int i = threadIdx.x; i < n * p.E; i += kThreads) {
            const int t_ = i / p.E, e = i - t_ * p.E;
            const float *z = p.part + (int64_t)(tok + t_) * p.E + e;
            float part[kMaxParts], v = 0.f;   // all loads at once
#pragma unroll
            for (int q = 0; q < kMaxParts; ++q)
                part[q] = q < p.kparts ? __ldcg(z + q * plane) : 0.f;
#pragma unroll
            for (int q = 0; q < kMaxParts; ++q)
                v += part[q];
            key[t_ * 2 * p.E + e] = __float_as_uint(v);
        }
        __syncthreads();
    }

    // Expert and weight of every assignment.  Up to 8 tokens every block finds them for itself, a
    // token a warp; with more, each token is one block's, and the blocks wait for one another.
    __device__ bool assign(uint16_t *expert, float *weight, int *s_ok)
    {
        uint32_t *key = reinterpret_cast<uint32_t *>(smem + p.sm_scratch);   // the ring is not in use yet
        float *bias = reinterpret_cast<float *>(key + (!kMany ? p.T : 1) * 2 * p.E);
        const float *use_bias = p.bias ? bias : nullptr;
        if (!kMany) {
            logits(0, p.T, key, bias);
            if (warp < p.T)
                route(p, key + warp * 2 * p.E, use_bias, expert + warp * p.k, weight + warp * p.k);
            __syncthreads();
        } else {
            for (int tok = blockIdx.x; tok < p.T; tok += gridDim.x) {
                logits(tok, 1, key, bias);
                if (warp == 0) {
                    route(p, key, use_bias, expert, weight);
                    for (int i = lane; i < p.k; i += 32) {
                        p.route_expert[tok * p.k + i] = expert[i];
                        p.route_weight[tok * p.k + i] = weight[i];
                    }
                }
                __syncthreads();
            }
            if (!grid_wait<kThreads>(p, 1, s_ok))
                return false;
            for (int a = threadIdx.x; a < p.T * p.k; a += kThreads)
                expert[a] = (uint16_t)__ldcg(p.route_expert + a);
            __syncthreads();
        }
        if (blockIdx.x == 0)
            for (int a = threadIdx.x; a < p.T * p.k; a += kThreads) {
                if (p.topk_weight)
                    p.topk_weight[a] = !kMany ? weight[a] : __ldcg(p.route_weight + a);
                if (p.expert_idx)
                    p.expert_idx[a] = expert[a];
            }
        return true;
    }

    // the active experts in order (one of more than 8 NT tokens several times, each time with as many),
    // and their columns; returns how many
    __device__ int columns(const uint16_t *expert)
    {
        uint16_t *act_ = reinterpret_cast<uint16_t *>(smem + p.sm_act);
        uint16_t *start_ = reinterpret_cast<uint16_t *>(smem + p.sm_start);
        uint16_t *cols_ = reinterpret_cast<uint16_t *>(smem + p.sm_cols);
        uint8_t *tokens_ = smem + p.sm_tokens;
        int *s_nact = reinterpret_cast<int *>(smem + p.sm_count);
        // in the ring, which is not in use yet: assignments of each expert, then its place among the
        // active ones; an assignment's place among its expert's
        uint16_t *count = reinterpret_cast<uint16_t *>(smem + p.sm_scratch), *place = count + p.E;
        const int n = p.T * p.k;
        for (int e = threadIdx.x; e < p.E; e += kThreads)
            count[e] = 0;
        if (!kMany)
            for (int i = threadIdx.x; i < min(n, p.E) * 8; i += kThreads)
                cols_[i] = 0xffffu;
        __syncthreads();
        if (warp == 0) {
            for (int a0 = 0; a0 < n; a0 += 32) {   // in order: an expert's columns are in token order
                const int a = a0 + lane, e = a < n ? expert[a] : -1;
                const uint32_t same = __match_any_sync(kFull, e);
                const int rank = __popc(same & ((1u << lane) - 1u)), before = a < n ? count[e] : 0;
                __syncwarp();   // every lane has read its count before the first of its expert's changes it
                if (a < n) {
                    place[a] = (uint16_t)(before + rank);
                    if (rank == 0)
                        count[e] = (uint16_t)(before + __popc(same));
                }
                __syncwarp();
            }
            int active = 0, at = 0;
            for (int e0 = 0; e0 < p.E; e0 += 32) {
                const int e = e0 + lane, c = e < p.E ? count[e] : 0, times = (c + 8 * NT - 1) / (8 * NT);
                int both = c << 16 | times, before = both;   // two sums in one word: at most 4096 of each
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(kFull, before, o);
                    before += lane >= o ? v : 0;
                }
                const int all = __shfl_sync(kFull, before, 31);
                before -= both;
                const int first = active + (before & 0xffff);
                for (int i = 0; i < times; ++i) {
                    act_[first + i] = (uint16_t)e;
                    start_[first + i] = (uint16_t)(at + (before >> 16) + i * 8 * NT);
                }
                if (c > 0)
                    count[e] = (uint16_t)first;
                at += all >> 16;
                active += all & 0xffff;
            }
            if (lane == 0) {
                start_[active] = (uint16_t)at;
                *s_nact = active;
            }
        }
        __syncthreads();
        for (int a = threadIdx.x; a < n; a += kThreads) {
            const int i = count[expert[a]], tok = a / p.k, c = !kMany ? i * 8 + tok : start_[i] + place[a];
            cols_[c] = (uint16_t)a;
            if (kMany)
                tokens_[c] = (uint8_t)tok;
        }
        __syncthreads();
        return *s_nact;
    }

    // this block's word of the first grid-wide wait, see there
    __device__ __forceinline__ void clear_word() const
    {
        if (threadIdx.x == 0)
            (blockIdx.x == 0 ? p.waits->go : p.waits->block[blockIdx.x]) = 0;
    }

    // a grid-wide wait has run out
    __device__ __forceinline__ void give_up() const
    {
        clear_word();
        if (threadIdx.x == 0)
            atomicOr(p.status, mrr_ws::kFlagTimeout);
    }

    // ------------------------------------------------------------ the two products

    // The down product with up to 8 tokens, whose columns are the tokens; with up to 4 (pairs) columns 4 .. 7 are
    // the second parts of h, else kOf parts come one after the other.
    template <int kOf, typename Take>
    __device__ __forceinline__ void down_few(int &buf, int *s_ok, Take take)
    {
        constexpr int kSteps = down_steps(kOf), kGroups = down_groups(kOf);
        const int token = p.pairs ? g % 4 : g;
        const uint32_t field = token < p.T ? field_of(token) : 127u;
        Cursor w;   // where the operands in `b` come from
        bool some = down_first() < down_items && first_chunk(w);
        Column c[kCols], c1[kCols];
        Tokens<kGroups, kOf> b;
        auto enter = [&](Column &to) {
            to = Column();
            const int a = column_of(w.expert, token);
            if (a >= 0) {
                to.v = p.h + kStored * ((int64_t)a * p.Ip + 8 * t) + (p.pairs && g >= 4 ? 8 : 0);
                to.tile = p.h_field + (int64_t)a * (p.Ip / 16) + t / 2;
            }
            to.field = field;
        };
        if (some) {
            enter(c1[0]);
            load_all<false>(b, c1, w.chunk * kDownK);
        }
        c[0].field = field;   // all that is still asked of the column whose operands are there
        // A token that did not choose an expert has zeros for it, which a NaN or an infinity in the expert's
        // weights would still reach: sums are taken over expert by expert, by the columns that chose it.
        const int pair_at = p.pairs ? 2 * t % 4 : 2 * t;
        for (int item = down_first(); item < down_items; item += gridDim.x) {
            float acc[2][NT][4] = {}, sum[4] = {};
            auto take_over = [&](int e) {
                uint32_t who = 0u;   // the two columns' assignments
                if (p.T > 1)
                    who = *reinterpret_cast<const uint32_t *>(cols + 8 * e + pair_at);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool chose = i % 2 ? who >> 16 != 0xffffu : (who & 0xffffu) != 0xffffu;
                    sum[i] += chose ? joined<kOf>(acc[0][0][i], acc[1][0][i]) : 0.f;
                    acc[0][0][i] = acc[1][0][i] = 0.f;
                }
            };
            for (bool more = some; more;) {
                const int at = take(), e = w.expert, k0 = w.chunk * kDownK;
                place_rows(p.w2, act[e] * p.H + item * 16, p.I, 0);
#pragma unroll
                for (int u = 0; u + 1 < kSteps; ++u)
                    multiply_all<false>(at, u * kGroups, 1, b, c, c1, 0, k0 + (u + 1) * kGroups * 32, acc,
                                        [&](int) { return Column(); });
                more = next_chunk(w);
                if (!more)   // the next item starts over
                    first_chunk(w);
                if (w.expert != e)
                    enter(c1[0]);
                multiply_all<false>(at, (kSteps - 1) * kGroups, 1, b, c, c1, 0, w.chunk * kDownK, acc,
                                    [&](int) { return Column(); });
                if (!more || (p.T > 1 && w.expert != e))   // one token chose all that are streamed
                    take_over(e);
            }
            put(red(buf), 0, sum, row);
            __syncthreads();
            if (threadIdx.x < 128) {
                const int r = threadIdx.x % 16, tok = threadIdx.x / 16, n = item * 16 + r;
                if (tok < p.T && n < p.H) {
                    float v = gather(red(buf), 0, r, tok);
                    if (p.pairs)
                        v = joined<2>(v, gather(red(buf), 0, r, tok + 4));
                    give(item, tok, r, v);
                }
            }
            if (splits() > 1)
                add_shares(item, s_ok);
            buf ^= 1;
        }
    }

    // The down product with more tokens: an expert's columns are the tokens that chose it.
    template <typename Take>
    __device__ __forceinline__ void down_many(int *s_ok, Take take)
    {
        constexpr int kSteps = down_steps(kParts), kGroups = down_groups(kParts);
        constexpr int kSumPitch = 17;   // [token][16 rows and a pad]
        float *mine = reinterpret_cast<float *>(smem + p.sm_red) + warp * p.T * kSumPitch;
        for (int item = down_first(); item < down_items; item += gridDim.x) {
            for (int i = lane; i < p.T * kSumPitch; i += 32)
                mine[i] = 0.f;
            __syncwarp();
            Cursor w;
            bool some = first_chunk(w);
            Column c[kCols], c1[kCols];
            Tokens<kGroups, kParts> b;
            auto enter = [&]() {   // the columns of expert w.expert
#pragma unroll
                for (int j = 0; j < kCols; ++j)
                    c1[j] = some && j < tiles_of(w.expert) ? h_column(w.expert, j) : Column();
            };
            enter();
            if (some)
                load_all<false>(b, c1, w.chunk * kDownK);
            while (some) {   // one share of an expert's K
                const int ai = w.expert, tiles = tiles_of(ai);
                place_rows(p.w2, act[ai] * p.H + item * 16, p.I, 0);
                float acc[2][NT][4] = {};
#pragma unroll
                for (int j = 0; j < kCols; ++j)
                    c[j] = c1[j];
                for (bool more = true; more;) {
                    const int at = take(), k0 = w.chunk * kDownK;
                    auto column = [&](int j) { return h_column(ai, j); };
#pragma unroll
                    for (int u = 0; u + 1 < kSteps; ++u)
                        multiply_all<false>(at, u * kGroups, tiles, b, c, c1, k0 + u * kGroups * 32,
                                            k0 + (u + 1) * kGroups * 32, acc, column);
                    more = ++w.chunk < w.last;
                    if (!more) {
                        w.part += down_stride();
                        some = enter_part(w);
                        enter();
                    }
                    multiply_all<false>(at, (kSteps - 1) * kGroups, tiles, b, c, c1, k0 + (kSteps - 1) * kGroups * 32,
                                        w.chunk * kDownK, acc, column);
                }
                const int first = start[ai], count = start[ai + 1] - first;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    if (j >= tiles)
                        break;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        if (8 * j + 2 * t + c < count) {
                            float *to = mine + tokens[first + 8 * j + 2 * t + c] * kSumPitch + row;
                            to[0] += joined<kParts>(acc[0][j][c], acc[1][j][c]);
                            to[8] += joined<kParts>(acc[0][j][2 + c], acc[1][j][2 + c]);
                        }
                }
                __syncwarp();   // the next share's columns are other lanes'
            }
            __syncthreads();
            const float *all = reinterpret_cast<const float *>(smem + p.sm_red);
            for (int i = threadIdx.x; i < 16 * p.T; i += kThreads) {
                const int r = i % 16, tok = i / 16, n = item * 16 + r;
                if (n >= p.H)
                    continue;
                float v = 0.f;
#pragma unroll
                for (int q = 0; q < kWarps; ++q)
                    v += all[(q * p.T + tok) * kSumPitch + r];
                give(item, tok, r, v);
            }
            if (splits() > 1)
                add_shares(item, s_ok);
            __syncthreads();
        }
    }

    __device__ void run()
    {
        int *s_ok = reinterpret_cast<int *>(smem + p.sm_count) + 1;
        if (blockIdx.x == 0 && threadIdx.x < 2) {
            p.waits->arrived[threadIdx.x] = 0;
            p.status[threadIdx.x] = 0;
        }
        if (kSplit && blockIdx.x == 0)
            for (int i = threadIdx.x; i < (p.H + 15) / 16; i += kThreads)
                p.split_count[i] = 0u;
        for (int tok = gridDim.x - 1 - blockIdx.x; tok < p.T; tok += gridDim.x)
            prepare_row(tok);
        for (int item = blockIdx.x; item < (p.E + 15) / 16 * p.kparts; item += gridDim.x)
            router_item(item);
        if (!grid_wait<kThreads>(p, 0, s_ok)) {
            give_up();
            return;
        }
        float *weight = reinterpret_cast<float *>(smem + p.sm_weight);
        uint16_t *expert = reinterpret_cast<uint16_t *>(smem);   // needed until the ring is
        if (!assign(expert, weight, s_ok)) {
            give_up();
            return;
        }
        sizes(columns(expert));

        tc::fence_to_async();   // the rings were scratch memory so far
        __syncthreads();
        Cursor next = first_unit();
        int slot = 0, fill_slot = 0, filled = 0;
        uint32_t parity = 0u;
        auto issue_next = [&]() {
            filled += next.phase < 2;
            issue(next, fill_slot);
            fill_slot = fill_slot + 1 == kStages ? 0 : fill_slot + 1;
        };
        // take the next stage: its copies have landed, and every lane is done with the one before
        auto take = [&]() {
            landed(slot, parity, next);
            issue_next();
            --filled;
            const int s = slot;
            slot = slot + 1 == kStages ? 0 : slot + 1;
            parity ^= slot == 0;
            return s;
        };
        // before leaving early: wait for what is in flight
        auto drain = [&]() {
            put_held();
            for (; filled > 0; --filled) {
                landed(slot, parity, next);
                slot = slot + 1 == kStages ? 0 : slot + 1;
                parity ^= slot == 0;
            }
            if (dead)
                settle();
        };
        for (int s = 0; s < kStages - 1; ++s)
            issue_next();

        int buf = 0;
        auto x_columns = [&](Column (&c)[kCols], int ai) {
#pragma unroll
            for (int j = 0; j < kCols; ++j)
                c[j] = j < tiles_of(ai) ? x_column(ai, j) : Column();
        };
        Column col[kCols], next_col[kCols];
        Tokens<kUpGroups> ahead;   // the next unit's operands
        if (up_first < up_items && up_begin < up_units) {
            x_columns(next_col, up_first / up_tiles);
            load_all<true>(ahead, next_col, up_begin * kUpK);
        }
        for (int item = up_first; item < up_items; item += up_stride) {
            const int ai = item / up_tiles, i0 = (item - ai * up_tiles) * 16, nt = tiles_of(ai);
            place_rows(p.w13, act[ai] * 2 * p.I + i0, p.H, p.I);
            float acc[2][NT][4] = {};
            for (int u = up_begin; u < up_units; u += up_step) {
                const int at = take();
                int k1 = (u + up_step) * kUpK;
                if (u + up_step >= up_units) {   // then comes the next item's first unit
                    k1 = up_begin * kUpK;
                    if (item + up_stride < up_items)
                        x_columns(next_col, (item + up_stride) / up_tiles);
                }
                multiply_all<true>(at, 0, nt, ahead, col, next_col, u * kUpK, k1, acc, [&](int j) { return x_column(ai, j); });
            }
            if (solo) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    if (j < nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            finish(weight, ai, i0, 8 * j + 2 * t + c, acc[0][j][c], acc[0][j][2 + c], acc[1][j][c], acc[1][j][2 + c]);
                continue;
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j >= nt)
                    break;
                put(red(buf), 0, acc[0][j], row);
                put(red(buf), 1, acc[1][j], row);
                __syncthreads();
                if (threadIdx.x < 128) {
                    const int r = threadIdx.x % 16, c = threadIdx.x / 16, a = column_of(ai, 8 * j + c);
                    if (a >= 0) {
                        const int tok = token_of(ai, 8 * j + c);
                        const float s = kMx ? p.x_scale[tok] : 1.f;
                        const float gate = gather(red(buf), 0, r, c) * s, upv = gather(red(buf), 1, r, c) * s;
                        // rows past I: what the copy brought there is another row's
                        float h = i0 + r < p.I ? gate / (1.f + expf(-gate)) * upv * (!kMany ? weight[a] : __ldcg(p.route_weight + a)) : 0.f;
                        if (kScaled) {
                            const uint32_t half = 0xffffu << (threadIdx.x & 16);
                            const uint32_t m = __reduce_max_sync(half, __float_as_uint(h) & 0x7fffffffu);
                            const uint32_t field = f16_scale_field(m);
                            h *= field_value(field);
                            if (r == 0) {
                                p.h_field[(int64_t)a * (p.Ip / 16) + i0 / 16] = (uint8_t)field;
                                atomicMax(p.h_max + tok, m);
                            }
                        }
                        store_h(a, i0 + r, h);
                    }
                }
                buf ^= 1;
            }
        }
        if (!grid_wait<kThreads>(p, 2, s_ok)) {
            drain();
            give_up();
            return;
        }
        clear_word();

        if (!kMany) {
            if (kParts == 2 && !p.pairs)
                down_few<kParts>(buf, s_ok, take);
            else
                down_few<1>(buf, s_ok, take);
        } else {
            down_many(s_ok, take);
        }
        if (dead) {   // every unit was waited for, or given up
            settle();
            if (lane == 0)
                atomicOr(p.status, mrr_ws::kFlagTimeout);
        }
    }
};

template <int DT, int WDT, int kRegime, bool kWide, bool kSplit>
__global__ void __launch_bounds__(32 * warps_of(WDT == MOE_MXFP4, kWide, kRegime), 1)
    layer_kernel(const __grid_constant__ Params p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    Layer<DT, WDT, kRegime, kWide, kSplit>(p, smem).run();
}

template <int DT, int WDT, int kRegime, bool kSplit>
static cudaError_t launch_one(const Params &p, const mrr_device::Info &info, int grid, size_t smem, cudaStream_t s)
{
    static std::atomic<uint64_t> allowed[2];
    const bool wide = p.w13_wide && p.w2_wide;
    auto kernel = wide ? layer_kernel<DT, WDT, kRegime, true, kSplit> : layer_kernel<DT, WDT, kRegime, false, kSplit>;
    const cudaError_t err = mrr_device::allow_smem(kernel, info, allowed[wide]);
    if (err != cudaSuccess)
        return err;
    void *args[] = {const_cast<Params *>(&p)};
    return cudaLaunchCooperativeKernel(reinterpret_cast<void *>(kernel), dim3(grid),
                                       dim3(32 * warps_of(WDT == MOE_MXFP4, wide, kRegime)), args, smem, s);
}

template <int DT, bool kSplit>
cudaError_t launch_dt(const Params &p, bool mx, int regime, const mrr_device::Info &info, int grid, size_t smem,
                      cudaStream_t s)
{
    if (regime == kFew)
        return mx ? launch_one<DT, MOE_MXFP4, kFew, kSplit>(p, info, grid, smem, s)
                  : launch_one<DT, DT, kFew, kSplit>(p, info, grid, smem, s);
    if (regime == kSpread)
        return mx ? launch_one<DT, MOE_MXFP4, kSpread, kSplit>(p, info, grid, smem, s)
                  : launch_one<DT, DT, kSpread, kSplit>(p, info, grid, smem, s);
    return launch_one<DT, DT, kDense, kSplit>(p, info, grid, smem, s);
}

// moe_layer_{bf16,f16}[_split].cu
using Launch = cudaError_t(const Params &p, bool mx, int regime, const mrr_device::Info &info, int grid, size_t smem,
                           cudaStream_t s);
Launch launch_bf16, launch_f16, launch_bf16_split, launch_f16_split;

}  // namespace moe_layer
