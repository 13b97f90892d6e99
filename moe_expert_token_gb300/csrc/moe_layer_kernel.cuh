// The kernel of the mixture-of-experts layer for a few tokens (include/moe_layer.h), for GB300
// (sm_103a).  moe_layer_{bf16,f16}.cu instantiate it, moe_layer.cu holds the host entry.
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
//    shared memory, filled with 16-byte asynchronous copies and waited for by that warp alone.
//    The ring runs on across items, and from the up product into the down product: the down
//    weights of the first items are in flight while the grid waits for h.
//  * A lane's 16-byte piece of a row feeds two matrix instructions: the order of k inside a group of
//    32 is free as long as both operands share it, so lane (g, t) holds elements 8t .. 8t+7.
//  * The grid waits twice: for the logits, and for h.  Between them every block computes the
//    routing of all tokens for itself, which costs less than a third wait.
//  * Up product: an item is 16 gate rows and the 16 up rows that belong to them, K split over the
//    warps, joined in shared memory; SwiGLU and the routing weight are applied there, in float32.
//  * Down product: an item is 16 output rows for all tokens; the warps split (expert, K) pairs.
// With up to 8 tokens the columns are the tokens themselves and the down product adds up all
// experts in registers; with more, an expert's columns are the tokens that chose it, and each
// warp adds them to its own sums in shared memory.  No sum depends on the order of anything but
// the sizes: results repeat bit for bit.
#pragma once

#include <math.h>

#include "moe_layer.h"
#include "mrr_gating.h"
#include "mx.cuh"
#include "ptx.cuh"
#include "ws_layout.h"

namespace moe_layer {

using namespace moe_mx;

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStages = 4;
constexpr int kUpRow = 128, kDownRow = 256;      // bytes of a row in a stage: 32 rows x 128, 16 rows x 256
constexpr uint64_t kWaitLimitNs = 2000000000ull;

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
    unsigned long long *flags;    // [2][grid], see grid_wait
    unsigned long long tag;
    float *part;                  // [kparts][T][E]
    uint16_t *xh;                 // [T][Hp]: x's rows as the products take them
    float *x_scale;               // [T]: what undoes their scaling
    uint32_t *h_max;              // [T]: float bits of the largest |h| of the token
    void *h;                      // [T k][Ip]
    int Hp, Ip, kparts;
    int x_wide, wr_wide, w13_wide, w2_wide, s13_wide, s2_wide;   // 16-byte (scales: 8-byte) copies possible
    // dynamic shared memory, byte offsets
    int sm_red, sm_y, sm_expert, sm_weight, sm_act, sm_start, sm_cols, sm_count;
};

__host__ __device__ constexpr int stage_bytes(bool mx) { return 4096 + (mx ? 256 : 0); }

template <int DT>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    if (DT == MOE_BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// asynchronous copies of 16 or 8 bytes; with ok false the destination is zeroed and src not read
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

__device__ __forceinline__ void copy8(uint32_t dst, const void *src, bool ok)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8 : 0) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// the power of two that takes the float with bits `amax` into [2^14, 2^15), so that it and all
// smaller ones fit float16 (1 where amax is 0, infinite or NaN), and its inverse
__device__ __forceinline__ float2 f16_scale(uint32_t amax)
{
    const int field = (int)(amax >> 23);
    if (amax == 0u || field == 255)
        return make_float2(1.f, 1.f);
    const int f = min(268 - field, 253);   // field <= 254: f >= 14
    return make_float2(__uint_as_float((uint32_t)f << 23), __uint_as_float((uint32_t)(254 - f) << 23));
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

// Eight codes to eight float16 values 2^14 times too small, as pairs (0, 4), (1, 5), (2, 6), (3, 7):
// a code's magnitude bits e e m are float16's low exponent bits and mantissa head (0.5 becomes a
// subnormal), so two codes 16 bits apart take four operations.
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t (&d)[4])
{
    d[0] = ((w << 12) & 0x80008000u) | ((w << 9) & 0x0e000e00u);
    d[1] = ((w << 8) & 0x80008000u) | ((w << 5) & 0x0e000e00u);
    d[2] = ((w << 4) & 0x80008000u) | ((w << 1) & 0x0e000e00u);
    d[3] = (w & 0x80008000u) | ((w >> 3) & 0x0e000e00u);
}

// ---------------------------------------------------------------- the grid-wide wait
//
// Block b writes the call's tag into its own word of `set` and waits until every block has.  The
// words need no initial value: tags are 64 random-looking bits, different for each call.  For a
// launch replayed from a graph, with the same tag: each block clears its word of set 1 before it
// arrives at set 0, and its word of set 0 once it is through set 1, so no word holds the tag
// before its block arrives.  The launch is cooperative (all blocks run at once); a wait that lasts
// kWaitLimitNs all the same gives up and returns false.
__device__ __forceinline__ bool grid_wait(const Params &p, int set, int *s_ok)
{
    unsigned long long *f = p.flags + (size_t)set * gridDim.x;
    __syncthreads();
    if (threadIdx.x == 0) {
        *s_ok = 1;
        __threadfence();
        asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(f + blockIdx.x), "l"(p.tag) : "memory");
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (int)gridDim.x; i += kThreads) {
        const uint64_t t0 = mrr::global_timer_ns();
        for (uint32_t it = 1;; ++it) {
            unsigned long long v;
            asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(f + i) : "memory");
            if (v == p.tag)
                break;
            if (it % 64 == 0 && mrr::global_timer_ns() - t0 > kWaitLimitNs) {
                *s_ok = 0;
                break;
            }
        }
    }
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

// The formulas of mrr_gating.h for token t; key: this warp's E words of shared memory.  Whatever the
// logits hold, the k experts are different and in range.
template <int DT>
__device__ void route(const Params &p, int t, uint32_t *key, uint16_t *expert, float *weight)
{
    const int lane = threadIdx.x % 32, E = p.E;
    const int64_t plane = (int64_t)p.T * E;
    const float *z = p.part + (int64_t)t * E;
    float mx = -INFINITY, sum = 0.f;
    for (int e = lane; e < E; e += 32) {
        float v = 0.f;
        for (int q = 0; q < p.kparts; ++q)
            v += z[q * plane + e];
        key[e] = __float_as_uint(v);
        mx = fmaxf(mx, v);
    }
    if (p.norm_type == 0) {
        mx = key_value(__reduce_max_sync(kFull, order_key(mx)));
        for (int e = lane; e < E; e += 32) {
            const float v = expf(__uint_as_float(key[e]) - mx);
            key[e] = __float_as_uint(v);
            sum += v;
        }
        sum = warp_sum(sum);
    }
    for (int e = lane; e < E; e += 32) {
        float v = __uint_as_float(key[e]);
        if (p.norm_type == 0)
            v = v / sum;
        else if (p.norm_type == 1)
            v = 1.f / (1.f + expf(-v));
        else
            v = v > 20.f ? v + log1pf(expf(-v)) : log1pf(expf(v));
        key[e] = order_key(p.bias ? v + load1<DT>(p.bias, e) : v);
    }
    __syncwarp();
    const int size = E / p.group_count;
    if (p.k_group < p.group_count) {
        // group scores; the groups are ranked over the lanes that hold them (32 at a time)
        uint32_t mine[MRR_GATE_MAX_EXPERTS / 32];   // key of group 32 i + lane
        const int rounds = (p.group_count + 31) / 32;
        for (int r = 0; r < rounds; ++r)
            mine[r] = 0u;
        for (int g = 0; g < p.group_count; ++g) {
            uint32_t a = 0u, b = 0u;   // this lane's two best of the group
            for (int e = g * size + lane; e < (g + 1) * size; e += 32) {
                const uint32_t v = key[e];
                b = max(b, min(a, v));
                a = max(a, v);
            }
            const uint32_t top = __reduce_max_sync(kFull, a);
            float s = key_value(top);
            if (p.select_mode == 1) {
                const bool first = __ffs(__ballot_sync(kFull, a == top)) - 1 == lane;
                s += key_value(__reduce_max_sync(kFull, first ? b : a));
            }
            if (g % 32 == lane)
                mine[g / 32] = order_key(s);
        }
        uint32_t kept[MRR_GATE_MAX_EXPERTS / 32];   // bit: group 32 i + lane is kept
        for (int r = 0; r < rounds; ++r)
            kept[r] = 0u;
        for (int i = 0; i < p.k_group; ++i) {
            uint32_t best = 0u;
            int at = 0;
            for (int r = 0; r < rounds; ++r)
                if (mine[r] > best) {
                    best = mine[r];
                    at = r;
                }
            const uint32_t top = __reduce_max_sync(kFull, best);
            const uint32_t g = __reduce_min_sync(kFull, best == top && best ? (uint32_t)(32 * at + lane) : 0xffffffffu);
            if ((int)(g % 32) == lane) {
                mine[g / 32] = 0u;
                kept[g / 32] = 1u;
            }
        }
        for (int g = 0; g < p.group_count; ++g)
            if (!(__ballot_sync(kFull, kept[g / 32]) >> (g % 32) & 1u))
                for (int e = g * size + lane; e < (g + 1) * size; e += 32)
                    key[e] = 0u;
        __syncwarp();
    }
    float total = 0.f;
    uint32_t best = 0u;
    int at = 0;
    auto scan = [&]() {
        best = 0u;
        for (int e = lane; e < E; e += 32)
            if (key[e] > best) {
                best = key[e];
                at = e;
            }
    };
    scan();
    for (int i = 0; i < p.k; ++i) {
        const uint32_t top = __reduce_max_sync(kFull, best);
        const uint32_t e = __reduce_min_sync(kFull, best == top && best ? (uint32_t)at : 0xffffffffu);
        const float s = key_value(top);
        total += s;
        if ((int)(e % 32) == lane) {
            expert[i] = (uint16_t)e;
            weight[i] = s;
            key[e] = 0u;
            scan();
        }
    }
    __syncwarp();
    for (int i = lane; i < p.k; i += 32)
        weight[i] = weight[i] / (total + p.eps) * p.rsf;
}

// ---------------------------------------------------------------- one warp's weight stream

// What comes next in a warp's stream: first its units of the up items of this block, then those of
// its down items.
struct Cursor {
    int phase, item, unit;   // phase 2: the stream is over
};

template <int DT, int WDT, int NT>
struct Layer {
    static constexpr bool kMx = WDT == MOE_MXFP4;
    static constexpr int MDT = kMx ? MOE_F16 : DT;            // the matrix instructions' type
    static constexpr bool kScaled = MDT == MOE_F16;           // h is float32 in memory, scaled when packed
    static constexpr int kStage = stage_bytes(kMx);
    static constexpr int kPerByte2 = kMx ? 4 : 1;             // elements in two bytes
    static constexpr int kUpK = kUpRow / 2 * kPerByte2, kDownK = kDownRow / 2 * kPerByte2;

    const Params &p;
    uint8_t *smem;
    uint32_t ring;               // this warp's stages
    int warp, lane, g, t;
    int nact, up_items, up_units, up_tiles, down_items, down_units, down_chunks;
    const uint16_t *act, *start, *cols;

    __device__ Layer(const Params &p_, uint8_t *sm) : p(p_), smem(sm)
    {
        warp = threadIdx.x / 32;
        lane = threadIdx.x % 32;
        g = lane / 4;
        t = lane % 4;
        ring = mrr::smem_addr(sm) + warp * kStages * kStage;
        act = reinterpret_cast<const uint16_t *>(sm + p.sm_act);
        start = reinterpret_cast<const uint16_t *>(sm + p.sm_start);
        cols = reinterpret_cast<const uint16_t *>(sm + p.sm_cols);
    }

    __device__ void sizes(int active)
    {
        nact = active;
        up_tiles = (p.I + 15) / 16;
        up_items = nact * up_tiles;
        up_units = (p.H + kUpK - 1) / kUpK;
        down_items = (p.H + 15) / 16;
        down_chunks = (p.I + kDownK - 1) / kDownK;
        down_units = nact * down_chunks;
    }

    // step to the first unit at or after c that exists
    __device__ __forceinline__ void settle(Cursor &c) const
    {
        if (c.phase == 0) {
            if (c.item < up_items && c.unit >= up_units) {
                c.unit = warp;
                c.item = c.unit < up_units ? c.item + gridDim.x : up_items;
            }
            if (c.item >= up_items)
                c = {1, (int)blockIdx.x, warp};
        }
        if (c.phase == 1) {
            if (c.item < down_items && c.unit >= down_units) {
                c.unit = warp;
                c.item = c.unit < down_units ? c.item + gridDim.x : down_items;
            }
            if (c.item >= down_items)
                c.phase = 2;
        }
    }

    // start the copies of unit c into stage `slot`: kRows rows of kRow bytes, 16-byte pieces
    // exchanged inside a row so that the reads below meet no bank twice
    template <int kRows, int kRow>
    __device__ __forceinline__ void fill(int slot, const void *w, const uint8_t *s, int64_t row0, int64_t second, int valid,
                                         int K, int chunk, bool wide, bool s_wide) const
    {
        constexpr int kPieces = kRow / 16;
        const int64_t row_bytes = kMx ? K / 2 : 2 * (int64_t)K;
        const int c = lane % kPieces;
        const int64_t off = (int64_t)chunk * kRow + c * 16;
        const uint32_t base = ring + slot * kStage;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = j * (32 / kPieces) + lane / kPieces;
            const bool ok = (r & 15) < valid && off < row_bytes;
            const int64_t row = row0 + (r & 15) + (kRows == 32 && r >= 16 ? second : 0);
            const uint32_t dst = base + r * kRow + ((kMx ? c ^ (r & 7) : c ^ ((r & 1) << 2)) << 4);
            const uint8_t *src = static_cast<const uint8_t *>(w) + row * row_bytes + off;
            if (wide) {
                copy16(dst, ok ? src : static_cast<const uint8_t *>(w), ok);
            } else {
                uint32_t v[4] = {0u, 0u, 0u, 0u};
                if (ok) {
                    if (kMx) {
                        for (int b = 0; b < 16; ++b)
                            if (off + b < row_bytes)
                                v[b / 4] |= (uint32_t)__ldg(src + b) << (8 * (b % 4));
                    } else {
                        for (int b = 0; b < 8; ++b)
                            if (off + 2 * b < row_bytes)
                                v[b / 2] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(src) + b) << (16 * (b % 2));
                    }
                }
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                             "r"(v[3])
                             : "memory");
            }
        }
        if (kMx) {   // 8 scale bytes a lane: row lane (32 rows of 8), or row lane / 2 (16 rows of 16)
            constexpr int kLanes = 32 / kRows;
            const int r = lane / kLanes;
            const int64_t srow = scale_row_bytes(K), soff = (int64_t)chunk * (8 * kLanes) + (lane % kLanes) * 8;
            const bool ok = (r & 15) < valid && soff < srow;
            const int64_t row = row0 + (r & 15) + (kRows == 32 && r >= 16 ? second : 0);
            const uint32_t dst = base + 4096 + lane * 8;
            const uint8_t *src = s + row * srow + soff;
            if (s_wide) {
                copy8(dst, ok ? src : s, ok);
            } else {
                uint32_t v[2] = {0u, 0u};
                if (ok)
                    for (int b = 0; b < 8; ++b)
                        if (soff + b < srow)
                            v[b / 4] |= (uint32_t)__ldg(src + b) << (8 * (b % 4));
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst), "r"(v[0]), "r"(v[1]) : "memory");
            }
        }
    }

    __device__ __forceinline__ void issue(Cursor &c, int slot) const
    {
        if (c.phase == 0) {
            const int ai = c.item / up_tiles, i0 = (c.item - ai * up_tiles) * 16;
            fill<32, kUpRow>(slot, p.w13, p.w13_s, (int64_t)act[ai] * 2 * p.I + i0, p.I, min(16, p.I - i0), p.H, c.unit,
                             p.w13_wide, p.s13_wide);
        } else if (c.phase == 1) {
            const int ai = c.unit / down_chunks, n0 = c.item * 16;
            fill<16, kDownRow>(slot, p.w2, p.w2_s, (int64_t)act[ai] * p.H + n0, 0, min(16, p.H - n0), p.I,
                               c.unit - ai * down_chunks, p.w2_wide, p.s2_wide);
        }
        copy_commit();
        if (c.phase < 2) {
            c.unit += kWarps;
            settle(c);
        }
    }

    __device__ __forceinline__ uint4 lds16(uint32_t at) const
    {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
        return v;
    }

    __device__ __forceinline__ uint32_t lds4(uint32_t at) const
    {
        uint32_t v;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
        return v;
    }

    __device__ __forceinline__ uint2 lds8(uint32_t at) const
    {
        uint2 v;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
        return v;
    }

    // The products of one stage: kTiles 16-row tiles against nt column tiles, groups of 32 k.
    // column(j, k): the 8 elements k .. k + 7 of this lane's column in tile j, packed.
    template <int kTiles, int kRow, typename Column>
    __device__ __forceinline__ void multiply(int slot, int K, int chunk, int nt, float (&acc)[kTiles][NT][4],
                                             Column column) const
    {
        constexpr int kGroups = kMx ? kRow / 16 : kRow / 64;
        const uint32_t base = ring + slot * kStage;
        const int k0 = chunk * kGroups * 32;
        uint2 sc[kMx ? kTiles : 1][2];   // scale bytes of rows g and g + 8, 8 groups at a time
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
            const int k = k0 + 32 * q;
            if (k >= K)
                break;
            if (kMx && q % 8 == 0)
#pragma unroll
                for (int m = 0; m < kTiles; ++m)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        sc[m][r] = lds8(base + 4096 + (16 * m + 8 * r + g) * (kRow / 16) + q);
            uint32_t a[kTiles][2][4];
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = 16 * m + 8 * r + g;
                    if (kMx) {
                        codes_to_half(lds4(base + row * kRow + ((q ^ (row & 7)) << 4) + 4 * t), a[m][r]);
                    } else {
                        const uint4 v = lds16(base + row * kRow + (((4 * q + t) ^ ((row & 1) << 2)) << 4));
                        a[m][r][0] = v.x, a[m][r][1] = v.y, a[m][r][2] = v.z, a[m][r][3] = v.w;
                    }
                }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j >= nt)
                    break;
                const uint4 b = column(j, k + 8 * t);
#pragma unroll
                for (int m = 0; m < kTiles; ++m) {
                    if (kMx) {
                        float d[4] = {0.f, 0.f, 0.f, 0.f};
                        mma<MDT>(d, a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1], b.x, b.y);
                        mma<MDT>(d, a[m][0][2], a[m][1][2], a[m][0][3], a[m][1][3], b.z, b.w);
                        const float s0 = e8m0_value((q % 8 < 4 ? sc[m][0].x : sc[m][0].y) >> (8 * (q % 4)) & 255u);
                        const float s1 = e8m0_value((q % 8 < 4 ? sc[m][1].x : sc[m][1].y) >> (8 * (q % 4)) & 255u);
                        acc[m][j][0] = fmaf(s0, d[0], acc[m][j][0]);
                        acc[m][j][1] = fmaf(s0, d[1], acc[m][j][1]);
                        acc[m][j][2] = fmaf(s1, d[2], acc[m][j][2]);
                        acc[m][j][3] = fmaf(s1, d[3], acc[m][j][3]);
                    } else {
                        mma<MDT>(acc[m][j], a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1], b.x, b.y);
                        mma<MDT>(acc[m][j], a[m][0][2], a[m][1][2], a[m][0][3], a[m][1][3], b.z, b.w);
                    }
                }
            }
        }
    }

    // assignment of column c of active expert ai, or -1.  Up to 8 tokens: column = token.
    __device__ __forceinline__ int column_of(int ai, int c) const
    {
        if (NT == 1) {
            const uint16_t a = cols[ai * 8 + c];
            return a == 0xffffu ? -1 : (int)a;
        }
        const int s = start[ai];
        return c < (int)start[ai + 1] - s ? (int)cols[s + c] : -1;
    }

    __device__ __forceinline__ int tiles_of(int ai) const
    {
        return NT == 1 ? 1 : ((int)start[ai + 1] - (int)start[ai] + 7) / 8;
    }

    // eight elements of h's row a as the matrix instructions take them
    __device__ __forceinline__ uint4 h8(int a, int k, float scale) const
    {
        if (a < 0 || k >= p.Ip)
            return make_uint4(0, 0, 0, 0);
        if (!kScaled)
            return *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.h) + (int64_t)a * p.Ip + k);
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p.h) + (int64_t)a * p.Ip + k);
        const float4 u = q[0], v = q[1];
        if (kMx)   // the order of codes_to_half
            return make_uint4(pack2<MDT>(u.x * scale, v.x * scale), pack2<MDT>(u.y * scale, v.y * scale),
                              pack2<MDT>(u.z * scale, v.z * scale), pack2<MDT>(u.w * scale, v.w * scale));
        return make_uint4(pack2<MDT>(u.x * scale, u.y * scale), pack2<MDT>(u.z * scale, u.w * scale),
                          pack2<MDT>(v.x * scale, v.y * scale), pack2<MDT>(v.z * scale, v.w * scale));
    }

    __device__ __forceinline__ float *red(int buf) const
    {
        return reinterpret_cast<float *>(smem + p.sm_red) + buf * (kWarps * 256);
    }

    // this warp's 16 x 8 partial sums into red[.][warp][tile][row][column]
    __device__ __forceinline__ void put(float *r, int tile, const float (&d)[4]) const
    {
        float *at = r + (warp * 2 + tile) * 128 + g * 8 + 2 * t;
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

    // ------------------------------------------------------------ before the first wait

    // x's row t as the products take it: 16-bit, zeros past H, scaled (kMx) and in their order
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
            const float2 s = f16_scale(*s_max);
            scale = s.x;
            if (threadIdx.x == 0)
                p.x_scale[tok] = s.y * 0x1p14f;   // and the codes' 2^14
            __syncthreads();
        } else if (threadIdx.x == 0) {
            p.x_scale[tok] = 1.f;
        }
        if (threadIdx.x == 0)
            p.h_max[tok] = 0u;
        for (int c = threadIdx.x; c < p.Hp / 8; c += kThreads) {
            uint4 v = load8_raw(p.x, tok, p.H, 8 * c, p.x_wide);
            if (kMx) {
                const float2 a = unpack2<DT>(v.x), b = unpack2<DT>(v.y), d = unpack2<DT>(v.z), e = unpack2<DT>(v.w);
                v = make_uint4(pack2<MDT>(a.x * scale, d.x * scale), pack2<MDT>(a.y * scale, d.y * scale),
                               pack2<MDT>(b.x * scale, e.x * scale), pack2<MDT>(b.y * scale, e.y * scale));
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
        float acc[NT][4] = {};
        for (int c = lo + warp; c < hi; c += kWarps) {
            uint4 a[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    a[r][q] = e0 + 8 * r + g < p.E ? load8_raw(p.wr, e0 + 8 * r + g, p.H, c * 128 + 32 * q + 8 * t, p.wr_wide)
                                                   : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
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
        for (int j = 0; j < NT; ++j) {
            if (8 * j >= p.T)
                break;
            put(red(j % 2), 0, acc[j]);
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

    // expert and weight of every assignment, the active experts in order, and their columns
    __device__ int routing()
    {
        uint16_t *expert = reinterpret_cast<uint16_t *>(smem + p.sm_expert);
        float *weight = reinterpret_cast<float *>(smem + p.sm_weight);
        uint16_t *act_ = reinterpret_cast<uint16_t *>(smem + p.sm_act);
        uint16_t *start_ = reinterpret_cast<uint16_t *>(smem + p.sm_start);
        uint16_t *cols_ = reinterpret_cast<uint16_t *>(smem + p.sm_cols);
        int *s_nact = reinterpret_cast<int *>(smem + p.sm_count);
        uint32_t *key = reinterpret_cast<uint32_t *>(smem) + warp * p.E;   // the ring is not in use yet
        uint16_t *count = reinterpret_cast<uint16_t *>(smem + kWarps * p.E * 4);
        for (int tok = warp; tok < p.T; tok += kWarps) {
            __syncwarp();
            route<DT>(p, tok, key, expert + tok * p.k, weight + tok * p.k);
        }
        __syncthreads();
        const int n = p.T * p.k;
        if (blockIdx.x == 0)
            for (int a = threadIdx.x; a < n; a += kThreads) {
                if (p.topk_weight)
                    p.topk_weight[a] = weight[a];
                if (p.expert_idx)
                    p.expert_idx[a] = expert[a];
            }
        for (int e = threadIdx.x; e < p.E; e += kThreads) {
            int c = 0;
            for (int a = 0; a < n; ++a)
                c += expert[a] == e;
            count[e] = (uint16_t)c;
        }
        __syncthreads();
        if (warp == 0) {
            int active = 0, at = 0;
            for (int e0 = 0; e0 < p.E; e0 += 32) {
                const int e = e0 + lane, c = e < p.E ? count[e] : 0;
                const uint32_t some = __ballot_sync(kFull, c > 0);
                int before = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(kFull, before, o);
                    before += lane >= o ? v : 0;
                }
                if (c > 0) {
                    const int i = active + __popc(some & ((1u << lane) - 1u));
                    act_[i] = (uint16_t)e;
                    start_[i] = (uint16_t)(at + before - c);
                }
                at += __shfl_sync(kFull, before, 31);
                active += __popc(some);
            }
            if (lane == 0) {
                start_[active] = (uint16_t)at;
                *s_nact = active;
            }
        }
        __syncthreads();
        const int active = *s_nact;
        for (int i = threadIdx.x; i < active; i += kThreads) {
            const int e = act_[i];
            int at = start_[i];
            if (NT == 1)
                for (int c = 0; c < 8; ++c)
                    cols_[i * 8 + c] = 0xffffu;
            for (int a = 0; a < n; ++a)
                if (expert[a] == e) {
                    if (NT == 1)
                        cols_[i * 8 + a / p.k] = (uint16_t)a;
                    else
                        cols_[at++] = (uint16_t)a;
                }
        }
        __syncthreads();
        return active;
    }

    // ------------------------------------------------------------ the two products

    __device__ void run()
    {
        int *s_ok = reinterpret_cast<int *>(smem + p.sm_count) + 1;
        if (threadIdx.x == 0)
            p.flags[gridDim.x + blockIdx.x] = 0;
        if (blockIdx.x == 0 && threadIdx.x < 2)
            p.status[threadIdx.x] = 0;
        for (int tok = gridDim.x - 1 - blockIdx.x; tok < p.T; tok += gridDim.x)
            prepare_row(tok);
        for (int item = blockIdx.x; item < (p.E + 15) / 16 * p.kparts; item += gridDim.x)
            router_item(item);
        if (!grid_wait(p, 0, s_ok)) {
            if (threadIdx.x == 0)
                atomicOr(p.status, mrr_ws::kFlagTimeout);
            return;
        }
        sizes(routing());
        const float *weight = reinterpret_cast<const float *>(smem + p.sm_weight);

        Cursor next = {0, (int)blockIdx.x, warp};
        settle(next);
        int slot = 0, fill_slot = 0;
        auto issue_next = [&]() {
            issue(next, fill_slot);
            fill_slot = fill_slot + 1 == kStages ? 0 : fill_slot + 1;
        };
        // take the next stage: its copies have landed, and every lane is done with the one before
        auto take = [&]() {
            copy_wait<kStages - 2>();
            __syncwarp();
            issue_next();
            const int s = slot;
            slot = slot + 1 == kStages ? 0 : slot + 1;
            return s;
        };
        for (int s = 0; s < kStages - 1; ++s)
            issue_next();

        int buf = 0;
        for (int item = blockIdx.x; item < up_items; item += gridDim.x) {
            const int ai = item / up_tiles, i0 = (item - ai * up_tiles) * 16, nt = tiles_of(ai);
            const uint16_t *row[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int a = j < nt ? column_of(ai, 8 * j + g) : -1;
                row[j] = a < 0 ? nullptr : p.xh + (int64_t)(a / p.k) * p.Hp;
            }
            float acc[2][NT][4] = {};
            for (int u = warp; u < up_units; u += kWarps)
                multiply<2, kUpRow>(take(), p.H, u, nt, acc, [&](int j, int k) {
                    return row[j] ? *reinterpret_cast<const uint4 *>(row[j] + k) : make_uint4(0, 0, 0, 0);
                });
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j >= nt)
                    break;
                put(red(buf), 0, acc[0][j]);
                put(red(buf), 1, acc[1][j]);
                __syncthreads();
                if (threadIdx.x < 128) {
                    const int r = threadIdx.x % 16, c = threadIdx.x / 16, a = column_of(ai, 8 * j + c);
                    if (a >= 0) {
                        const int tok = a / p.k;
                        const float s = kMx ? p.x_scale[tok] : 1.f;
                        const float gate = gather(red(buf), 0, r, c) * s, upv = gather(red(buf), 1, r, c) * s;
                        const float h = gate / (1.f + expf(-gate)) * upv * weight[a];
                        if (kScaled) {
                            static_cast<float *>(p.h)[(int64_t)a * p.Ip + i0 + r] = h;
                            const uint32_t half = 0xffffu << (threadIdx.x & 16);
                            const uint32_t m = __reduce_max_sync(half, __float_as_uint(h) & 0x7fffffffu);
                            if (r == 0)
                                atomicMax(p.h_max + tok, m);
                        } else {
                            store1<MOE_BF16>(p.h, (int64_t)a * p.Ip + i0 + r, h);
                        }
                    }
                }
                buf ^= 1;
            }
        }
        if (!grid_wait(p, 1, s_ok)) {
            copy_wait<0>();
            if (threadIdx.x == 0)
                atomicOr(p.status, mrr_ws::kFlagTimeout);
            return;
        }
        if (threadIdx.x == 0)
            p.flags[blockIdx.x] = 0;

        // what the matrix instructions' sums are multiplied by for token tok, and h before them
        auto h_scale = [&](int tok) { return kScaled ? f16_scale(__ldcg(p.h_max + tok)) : make_float2(1.f, 1.f); };
        if (NT == 1) {
            const float scale = g < p.T ? h_scale(g).x : 1.f;
            for (int item = blockIdx.x; item < down_items; item += gridDim.x) {
                float acc[1][NT][4] = {};
                for (int u = warp; u < down_units; u += kWarps) {
                    const int ai = u / down_chunks, a = column_of(ai, g);
                    multiply<1, kDownRow>(take(), p.I, u - ai * down_chunks, 1, acc,
                                          [&](int, int k) { return h8(a, k, scale); });
                }
                put(red(buf), 0, acc[0][0]);
                __syncthreads();
                if (threadIdx.x < 128) {
                    const int r = threadIdx.x % 16, tok = threadIdx.x / 16, n = item * 16 + r;
                    if (tok < p.T && n < p.H)
                        store1<DT>(p.y, (int64_t)tok * p.H + n,
                                   gather(red(buf), 0, r, tok) * h_scale(tok).y * (kMx ? 0x1p14f : 1.f));
                }
                buf ^= 1;
            }
        } else {
            constexpr int kPitch = 17;   // [token][16 rows and a pad]
            float *mine = reinterpret_cast<float *>(smem + p.sm_y) + warp * p.T * kPitch;
            for (int item = blockIdx.x; item < down_items; item += gridDim.x) {
                for (int i = lane; i < p.T * kPitch; i += 32)
                    mine[i] = 0.f;
                __syncwarp();
                for (int u = warp; u < down_units; u += kWarps) {
                    const int ai = u / down_chunks, nt = tiles_of(ai);
                    int a[NT];
                    float scale[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        a[j] = j < nt ? column_of(ai, 8 * j + g) : -1;
                        scale[j] = kScaled && a[j] >= 0 ? h_scale(a[j] / p.k).x : 1.f;
                    }
                    float acc[1][NT][4] = {};
                    multiply<1, kDownRow>(take(), p.I, u - ai * down_chunks, nt, acc,
                                          [&](int j, int k) { return h8(a[j], k, scale[j]); });
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        if (j >= nt)
                            break;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int q = column_of(ai, 8 * j + 2 * t + c);
                            if (q >= 0) {
                                float *at = mine + (q / p.k) * kPitch + g;
                                at[0] += acc[0][j][c];
                                at[8] += acc[0][j][2 + c];
                            }
                        }
                    }
                }
                __syncthreads();
                const float *all = reinterpret_cast<const float *>(smem + p.sm_y);
                for (int i = threadIdx.x; i < 16 * p.T; i += kThreads) {
                    const int r = i % 16, tok = i / 16, n = item * 16 + r;
                    if (n >= p.H)
                        continue;
                    float v = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w)
                        v += all[(w * p.T + tok) * kPitch + r];
                    store1<DT>(p.y, (int64_t)tok * p.H + n, v * h_scale(tok).y * (kMx ? 0x1p14f : 1.f));
                }
                __syncthreads();
            }
        }
        copy_wait<0>();
    }
};

template <int DT, int WDT, int NT>
__global__ void __launch_bounds__(kThreads, 1) layer_kernel(const __grid_constant__ Params p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    Layer<DT, WDT, NT>(p, smem).run();
}

template <int DT, int WDT, int NT>
cudaError_t launch_one(const Params &p, int grid, size_t smem, cudaStream_t s)
{
    auto kernel = layer_kernel<DT, WDT, NT>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess)
        return err;
    void *args[] = {const_cast<Params *>(&p)};
    return cudaLaunchCooperativeKernel(reinterpret_cast<void *>(kernel), dim3(grid), dim3(kThreads), args, smem, s);
}

template <int DT>
cudaError_t launch_dt(const Params &p, bool mx, int grid, size_t smem, cudaStream_t s)
{
    if (p.T <= 8)
        return mx ? launch_one<DT, MOE_MXFP4, 1>(p, grid, smem, s) : launch_one<DT, DT, 1>(p, grid, smem, s);
    return mx ? launch_one<DT, MOE_MXFP4, 8>(p, grid, smem, s) : launch_one<DT, DT, 8>(p, grid, smem, s);
}

cudaError_t launch_bf16(const Params &p, bool mx, int grid, size_t smem, cudaStream_t s);
cudaError_t launch_f16(const Params &p, bool mx, int grid, size_t smem, cudaStream_t s);

}  // namespace moe_layer
