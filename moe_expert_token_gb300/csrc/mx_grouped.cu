// The experts' product on expert-major MXFP4 rows (include/moe_mx.h), for GB300 (sm_103a).
//
// y[r, n] = sum_k x[r, k] w[e(r), n, k]; gated: silu(y_gate) * y_up; times row_weight.
//
// Both operands stay in 4 bits up to the tensor cores: tcgen05.mma kind::mxf4 multiplies e2m1 codes
// and applies the e8m0 scales of 32-element blocks itself, with float32 sums in tensor memory.
//
//  * Weights are the 128-row operand and token rows the columns, so an expert with few rows pads
//    16 columns and not 128 rows, and a lane of the result holds one output feature: 32 lanes are
//    one 32-block of an MXFP4 result, and a gate and its up value meet in the same lane.
//  * A tile is two 128-row weight tiles (gated: the gate rows and their up rows; else neighbours), or
//    one where that fills the blocks more evenly, by up to 192 token rows of one expert, K in steps
//    of 256 (128 bytes a row).  An expert's rows are split evenly over its tiles, in multiples of 16.
//  * One persistent block an SM.  Warp 0 issues the tiled bulk copies of codes, warp 1 the matrix
//    instructions, warps 12-15 bring the scales, warps 4-11 turn finished sums into results while
//    the next tile's stages are being filled.
//  * Scales go from global memory through shared memory, where they change order, into tensor memory
//    by the scale warps' own stores.  The tensor pipe's copy instruction would do the last leg, but
//    it holds up the matrix instructions behind it: 8 copies a step took a third of the kernel's time.
//  * Neighbouring blocks work on the token tiles of the same weights, which so come from HBM once.
//
// Measured, gated, 32 experts of 7168 x 2048: 512 rows 83 us, the weights' 499 MB at 6.0 TB/s, bound by HBM;
// 16384 rows 201 us, 962 GFLOP at 4.8 PFLOP/s, bound by the copies from L2 into shared memory (57 KB a
// step of 25 MFLOP), the tensor pipe (53 % active) and the results, which are written between tiles.
//
// Every wait is bounded: one that lasts two seconds sets a flag, all roles leave, copies in flight
// are waited for, tensor memory is freed, and mrr_v2_read_status reports MRR_ERR_TIMEOUT.
#include <cuda.h>

#include "device_info.h"
#include "mx.cuh"
#include "tc.cuh"
#include "ws_layout.h"

using namespace moe_mx;

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 512;
constexpr int kEpilogueWarp = 4, kEpilogueWarps = 8, kScaleWarp = 12;
constexpr int kRowTile = 128;            // weight rows of one matrix instruction
constexpr int kStepBytes = 128;          // bytes of a row in a stage: 256 elements
__host__ __device__ constexpr int box_rows(int i) { return i < 2 ? 32 << i : 64 * i; }   // token rows of a copy: 32, 64, 128, 192
constexpr int kMaxStages = 8;
constexpr int kColumns = 512;            // all of tensor memory
constexpr int kMaxExperts = 4096;
constexpr int kTurnPitch = 36;           // floats: 16-byte reads of rows and 4-byte writes of columns, no bank twice
constexpr int kFewRows = 24;             // so many rows an expert, on average, or fewer: weights' bytes are what counts
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// The barriers, for tests that let a wait run out: one of a kind expects an arrival that never comes.
enum Barrier { kNone, kFullStage, kEmptyStage, kFullSums, kEmptySums };

struct Params {
    const uint8_t *scales, *w_scales;
    int A, K, E, N, counts_i64, counts_prefix, gated, out_dt;
    const void *counts;
    const float *row_weight;
    void *out;
    uint8_t *out_scales;
    uint32_t *status;
    int tokens;        // most token rows of a tile (64 or 192)
    int stages, sums;  // ring stages; sets of sums in tensor memory (1 or 2)
    int align, w_align;    // of scale rows: 32, 16, 8 or 2 bytes
    int out_wide;          // 16-bit and MXFP4 rows can be written so many bytes at a time: 32, 8, or 0 (less)
    int sm_stage, sm_tables, sm_scales, sm_turn;
    uint64_t wait_ns;  // limit of each wait
    int short_of;      // a Barrier, else kNone
};

struct Maps {
    CUtensorMap w, x[4];   // x: boxes of box_rows(i) rows
};

struct Tile {
    int expert, feature, row, rows, columns;   // columns: rows rounded up to 16
};

__host__ __device__ constexpr int groups_of(int tokens) { return (tokens + 127) / 128; }
__host__ __device__ constexpr int stage_bytes(int halves, int tokens)
{
    return (halves * kRowTile + tokens) * kStepBytes;
}

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], sums_full[2], sums_empty[2], drained;
    long long scan_rows[kThreads / 32];
    int scan_tiles[kThreads / 32];
    uint32_t tmem;
    int abort, bad;
};

// Wait for a phase of `bar`, by a whole warp, which stays together: false for all of it where a lane has
// given up, after p.wait_ns or because another warp has.
__device__ __forceinline__ bool wait(const Params &p, Shared *sh, uint64_t *bar, uint32_t parity)
{
    bool there = true;
    uint64_t t0 = 0;   // the timer is slow to read: not before a wait has become a long one
    for (uint32_t it = 1; !mrr::mbar_try_wait(mrr::smem_addr(bar), parity); ++it)
        if (it % 1024 == 0) {
            const uint64_t now = mrr::global_timer_ns();
            if (t0 == 0)
                t0 = now;
            else if (now - t0 > p.wait_ns)
                *reinterpret_cast<volatile int *>(&sh->abort) = 1;
            if (*reinterpret_cast<volatile int *>(&sh->abort)) {
                there = false;
                break;
            }
        }
    return __all_sync(kFull, there);
}

// Row and tile prefixes of the experts, into tables[0 .. E] and tables[E + 1 .. 2 E + 1]; flags of bad
// counts.  Every thread sums a run of experts, then the runs are scanned over the block.
__device__ int scan_counts(const Params &p, Shared *sh, int *tables)
{
    const int per = (p.E + kThreads - 1) / kThreads, lo = min(p.E, (int)threadIdx.x * per), hi = min(p.E, lo + per);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    auto at = [&](int e) {
        return p.counts_i64 ? (long long)__ldg(static_cast<const long long *>(p.counts) + e)
                            : (long long)__ldg(static_cast<const int *>(p.counts) + e);
    };
    if (threadIdx.x == 0)
        sh->bad = 0;
    __syncthreads();
    long long rows = 0;
    int tiles = 0, bad = 0;
    for (int e = lo; e < hi; ++e) {
        const long long v = at(e), c = p.counts_prefix && e > 0 ? v - at(e - 1) : v;
        if (c < 0 || (p.counts_prefix && v < 0))
            bad |= mrr_ws::kFlagNonPos;
        else if (c > p.A || v > p.A)
            bad |= mrr_ws::kFlagSum;
        else {
            rows += c;
            tiles += (int)((c + p.tokens - 1) / p.tokens);
        }
    }
    // a run's rows are at most 8 A < 2^34: cap them, a sum above A is refused below
    int r = (int)min(rows, (long long)p.A + 1 > 0x7fffffffll ? 0x7fffffffll : (long long)p.A + 1), t = tiles;
    if (rows > p.A)
        bad |= mrr_ws::kFlagSum;
    if (bad)
        atomicOr(&sh->bad, bad);
    __syncthreads();
    if (sh->bad)   // no sum is formed of counts that do not fit
        return sh->bad & mrr_ws::kFlagNonPos ? mrr_ws::kFlagNonPos : mrr_ws::kFlagSum;
    // the sum over the block may pass 2^31 where single runs do not: scan in 64 bits
    long long rs = r;
    int ts = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(kFull, rs, o);
        const int b = __shfl_up_sync(kFull, ts, o);
        if (lane >= o) {
            rs += a;
            ts += b;
        }
    }
    if (lane == 31) {
        sh->scan_rows[warp] = rs;
        sh->scan_tiles[warp] = ts;
    }
    __syncthreads();
    long long row0 = rs - r, total = 0;
    int tile0 = ts - t;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) {
            row0 += sh->scan_rows[w];
            tile0 += sh->scan_tiles[w];
        }
        total += sh->scan_rows[w];
    }
    if (total != p.A)
        return mrr_ws::kFlagSum;
    for (int e = lo; e < hi; ++e) {
        tables[e] = (int)row0;
        tables[p.E + 1 + e] = tile0;
        const int c = (int)(p.counts_prefix && e > 0 ? at(e) - at(e - 1) : at(e));
        row0 += c;
        tile0 += (c + p.tokens - 1) / p.tokens;
    }
    if (hi == p.E && lo < hi) {
        tables[p.E] = (int)row0;
        tables[2 * p.E + 1] = tile0;
    }
    __syncthreads();
    return 0;
}

// tile `index` of an expert's rows by `width` output features
__device__ __forceinline__ Tile tile_at(const Params &p, const int *tables, int features, int width, long long index)
{
    const int *rows = tables, *tiles = tables + p.E + 1;
    int lo = 0, hi = p.E - 1;   // the last expert whose first tile is at or before index (one that has tiles)
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if ((long long)tiles[mid] * features <= index)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int n = tiles[lo + 1] - tiles[lo], count = rows[lo + 1] - rows[lo];
    const int q = (int)(index - (long long)tiles[lo] * features), f = q / n, i = q - f * n;
    const int share = (((count + n - 1) / n) + 15) & ~15;
    Tile t;
    t.expert = lo;
    t.feature = f * width;
    t.row = rows[lo] + i * share;
    t.rows = min(share, count - i * share);
    t.columns = (t.rows + 15) & ~15;
    return t;
}

// Scale bytes of 32 blocks of row `row` from block b0, four steps' worth: a whole 32-byte sector
// where rows are aligned to one (8 bytes a step would be fetched four times over).  align: 32, 16, 8
// or 2, what rows and base are aligned to.  Blocks at or past `blocks` read 0: their codes are zeros, and a
// scale of 2^-127 keeps them so.
__device__ __forceinline__ void scales32(uint32_t (&v)[8], const uint8_t *s, int64_t row, int64_t row_bytes, int b0,
                                         int blocks, int align)
{
    const uint8_t *at = s + row * row_bytes + b0;
    const int left = blocks - b0;
    if (align == 32 && left > 0) {   // b0 is a multiple of 32 and rows of 16 or 32 bytes: what is loaded lies inside the row
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "l"(at));
    } else if (align >= 16) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 q = 16 * i < left ? __ldg(reinterpret_cast<const uint4 *>(at) + i) : make_uint4(0, 0, 0, 0);
            v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
        }
    } else if (align == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint2 q = 8 * i < left ? __ldg(reinterpret_cast<const uint2 *>(at) + i) : make_uint2(0, 0);
            v[2 * i] = q.x, v[2 * i + 1] = q.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // pairs are whole: a row holds ceil(K / 64) of them
            const uint32_t lo = 4 * i < left ? __ldg(reinterpret_cast<const uint16_t *>(at) + 2 * i) : 0u;
            const uint32_t hi = 4 * i + 2 < left ? __ldg(reinterpret_cast<const uint16_t *>(at) + 2 * i + 1) : 0u;
            v[i] = lo | hi << 16;
        }
    }
    if (left < 32)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] &= left >= 4 * i + 4 ? kFull : left > 4 * i ? (1u << (8 * (left - 4 * i))) - 1u : 0u;
}

// named barrier `id` of `threads` threads: true for all of them if `failed` is for any
__device__ __forceinline__ bool any_of(int id, int threads, bool failed)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                 "barrier.cta.red.or.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)failed), "r"(id), "r"(threads)
                 : "memory");
    return r != 0u;
}

// silu(g) u = g u / (1 + exp(-g)).  Results of 16 bits or fewer take the hardware's base-2 exponential and
// reciprocal, 6 instructions where expf and a division are some 20: the epilogue is bound by them, and
// the tile after it waits.  The error, |g| 2^-24 from rounding g log2(e) and a few 2^-23, is far below
// theirs.  Extremes: g = -inf gives -inf * 0 = NaN as the formula does, other large |g| 0 or g u.
template <int kOut>
__device__ __forceinline__ float swiglu(float g, float u)
{
    if constexpr (kOut == MOE_F32) {
        return __fdividef(g, 1.f + expf(-g)) * u;
    } else {
        float e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
        return g * r * u;
    }
}

// 16 columns of a feature a lane to 16 features of a column for each two lanes, through the warp's
// 16 x kTurnPitch floats of shared memory
__device__ __forceinline__ void turn_over(float *turn, int lane, const float (&y)[16], float (&v)[16])
{
#pragma unroll
    for (int j = 0; j < 16; ++j)
        turn[j * kTurnPitch + lane] = y[j];
    __syncwarp();
    const float4 *from = reinterpret_cast<const float4 *>(turn + lane / 2 * kTurnPitch + lane % 2 * 16);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float4 f = from[c];
        v[4 * c] = f.x, v[4 * c + 1] = f.y, v[4 * c + 2] = f.z, v[4 * c + 3] = f.w;
    }
    __syncwarp();
}

// Results of 16 columns (token rows row .. row + rows - 1) of one output feature a lane: n0 + lane.
// They are turned over first, so that a lane stores 32 bytes of a row (16-bit results) or 8 (codes), and a
// block's maximum and scale are found by two lanes and not by 32.
template <int kOut>
__device__ __forceinline__ void store16(const Params &p, int64_t row, int rows, int n0, int lane, float *turn,
                                        const float (&y)[16])
{
    const int n = n0 + lane;
    if constexpr (kOut == MOE_MXFP4) {   // 32 lanes are one block; N is a multiple of 32
        if (n0 >= p.N)
            return;
        float v[16];
        turn_over(turn, lane, y, v);
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(kFull, m, 1));
        const uint32_t s = scale_byte(m);
        const float r = inverse_scale(s);
        float lo[8], hi[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            lo[j] = v[j] * r, hi[j] = v[8 + j] * r;
        const uint32_t w[2] = {encode8(lo), encode8(hi)};
        const int i = lane / 2;
        if (i < rows) {
            uint8_t *q = static_cast<uint8_t *>(p.out) + (row + i) * (p.N / 2) + n0 / 2 + lane % 2 * 8;
            if (p.out_wide) {
                *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
            } else {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    q[c] = (uint8_t)(w[c / 4] >> (8 * (c % 4)));
            }
            if (lane % 2 == 0) {
                uint8_t *so = p.out_scales + (row + i) * scale_row_bytes(p.N) + n0 / 32;
                so[0] = (uint8_t)s;
                if (n0 / 32 % 2 == 0 && n0 + 32 >= p.N)
                    so[1] = 127;
            }
        }
    } else if (kOut != MOE_F32 && p.out_wide) {   // N is a multiple of 4
        float v[16];
        turn_over(turn, lane, y, v);
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = pack2<kOut>(v[2 * j], v[2 * j + 1]);
        const int f = n0 + lane % 2 * 16;   // this lane's first feature
        uint16_t *q = static_cast<uint16_t *>(p.out) + (row + lane / 2) * p.N + f;
        if (lane / 2 < rows && f < p.N) {
            if (p.out_wide == 32) {
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(q), "r"(w[0]), "r"(w[1]),
                             "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                             : "memory");
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (f + 4 * j < p.N)
                        reinterpret_cast<uint2 *>(q)[j] = make_uint2(w[2 * j], w[2 * j + 1]);
            }
        }
    } else {
        if (n >= p.N)
            return;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (j < rows)
                store1<kOut>(p.out, (row + j) * p.N + n, y[j]);
    }
}

// kTiles: 128-row weight tiles of a tile of results.  2: the gate rows and their up rows, or neighbours.
// 1: 64 gate rows and their 64 up rows, or 128 rows.
template <bool kGated, int kOut, int kTiles>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared *sh = reinterpret_cast<Shared *>(smem);
    int *tables = reinterpret_cast<int *>(smem + p.sm_tables);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    const int bad = scan_counts(p, sh, tables);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.status[0] = (uint32_t)bad;
        p.status[1] = 0;
    }
    if (bad)
        return;
    constexpr int mats = kGated ? 2 : 1, kFeatures = kTiles * kRowTile / mats;
    constexpr bool kMixed = kGated && kTiles == 1;   // gate and up rows in one tile
    const int features = (p.N + kFeatures - 1) / kFeatures;
    const long long total = (long long)tables[2 * p.E + 1] * features;
    if ((long long)blockIdx.x >= total)
        return;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mrr::mbar_init(mrr::smem_addr(&sh->full[s]), 1 + 4 + (p.short_of == kFullStage));   // the copies' thread, four scale warps
            mrr::mbar_init(mrr::smem_addr(&sh->empty[s]), 1 + (p.short_of == kEmptyStage));
        }
        for (int b = 0; b < 2; ++b) {
            mrr::mbar_init(mrr::smem_addr(&sh->sums_full[b]), 1 + (p.short_of == kFullSums));
            mrr::mbar_init(mrr::smem_addr(&sh->sums_empty[b]), kEpilogueWarps + (p.short_of == kEmptySums));
        }
        mrr::mbar_init(mrr::smem_addr(&sh->drained), 1);
        sh->abort = 0;
        mrr::mbar_init_fence();
        tc::prefetch_map(&maps.w);
        for (const CUtensorMap &m : maps.x)
            tc::prefetch_map(&m);
    }
    if (warp == 1)
        tc::alloc(mrr::smem_addr(&sh->tmem), kColumns);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&sh->tmem);

    const int steps = (p.K + 255) / 256, groups = groups_of(p.tokens);
    const uint32_t stage0 = mrr::smem_addr(smem) + p.sm_stage;
    const uint32_t stage_size = stage_bytes(kTiles, p.tokens);
    const uint32_t scale_columns = 8 * kTiles + 8 * groups, sums_columns = kTiles * p.tokens;
    const uint32_t off_x = kTiles * kRowTile * kStepBytes;
    auto next_stage = [&](int &stage, uint32_t &parity) {
        if (++stage == p.stages) {
            stage = 0;
            parity ^= 1u;
        }
    };

    // Warps 0 and 1 run their loops as whole warps, one lane issuing: so the compiler keeps what an
    // instruction takes in uniform registers.  As one thread's code each matrix instruction cost 84
    // cycles to issue, as many as it runs.
    if (warp == 0) {   // codes
        const bool leader = tc::elect();
        int stage = 0;
        uint32_t parity = 1u;
        bool ok = true;
        for (long long i = blockIdx.x; ok && i < total; i += gridDim.x) {
            const Tile t = tile_at(p, tables, features, kFeatures, i);
            const int w_row = tc::uniform(t.expert * mats * p.N + t.feature), x_row = tc::uniform(t.row);
            const int second = kGated ? p.N : kRowTile;
            // one copy for all token rows: the smallest box that holds them
            const int box = tc::uniform(t.columns <= 32 ? 0 : t.columns <= 64 ? 1 : t.columns <= 128 ? 2 : 3);
            const CUtensorMap *x_map = &maps.x[box];
            const uint32_t bytes = (kTiles * kRowTile + box_rows(box)) * kStepBytes;
            for (int k = 0; k < steps; ++k) {
                if (!(ok = wait(p, sh, &sh->empty[stage], parity)))
                    break;
                const uint32_t at = stage0 + stage * stage_size, bar = mrr::smem_addr(&sh->full[stage]);
                if (leader) {
                    mrr::mbar_arrive_expect_tx(bar, bytes);
                    tc::load_box(at, &maps.w, k * kStepBytes, w_row, bar);
                    if (kTiles == 2 || kMixed)
                        tc::load_box(at + (kMixed ? kRowTile / 2 : kRowTile) * kStepBytes, &maps.w, k * kStepBytes,
                                     w_row + second, bar);
                    tc::load_box(at + off_x, x_map, k * kStepBytes, x_row, bar);
                }
                __syncwarp();
                next_stage(stage, parity);
            }
        }
    } else if (warp == 1) {   // matrix instructions
        const bool leader = tc::elect();
        int stage = 0, set = 0;
        uint32_t parity = 0u, set_parity = 1u;
        bool ok = true;
        const uint32_t scales0 = tmem + p.sums * sums_columns;
        for (long long i = blockIdx.x; ok && i < total; i += gridDim.x) {
            const Tile t = tile_at(p, tables, features, kFeatures, i);
            if (!(ok = wait(p, sh, &sh->sums_empty[set], set_parity)))
                break;
            tc::fence_after();
            const uint32_t d = tmem + set * sums_columns;
            const uint32_t columns = tc::uniform(t.columns);
            const uint32_t instr[2] = {tc::mxf4_instr(columns, 0), tc::mxf4_instr(columns, 1)};
            for (int k = 0; k < steps; ++k) {
                if (!(ok = wait(p, sh, &sh->full[stage], parity)))
                    break;
                tc::fence_after();
                const uint32_t at = stage0 + stage * stage_size;
                const uint32_t sfa = scales0 + stage * scale_columns, sfb = sfa + 8 * kTiles;
                const uint64_t w0 = tc::desc_swizzle128(at), w1 = tc::desc_swizzle128(at + kRowTile * kStepBytes);
                const uint64_t x = tc::desc_swizzle128(at + off_x);
                if (leader) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {   // 64 elements (past K: zeros): 32 bytes further along the rows
                        const uint32_t half = j / 2;
                        tc::mma_mxf4(d, w0 + 2 * j, x + 2 * j, instr[j % 2], sfa + 4 * half, sfb + 4 * groups * half,
                                     k > 0 || j > 0);
                        if (kTiles == 2)
                            tc::mma_mxf4(d + p.tokens, w1 + 2 * j, x + 2 * j, instr[j % 2], sfa + 8 + 4 * half,
                                         sfb + 4 * groups * half, k > 0 || j > 0);
                    }
                    tc::commit(mrr::smem_addr(&sh->empty[stage]));
                    if (k + 1 == steps)
                        tc::commit(mrr::smem_addr(&sh->sums_full[set]));
                }
                __syncwarp();
                next_stage(stage, parity);
            }
            if (++set == p.sums) {
                set = 0;
                set_parity ^= 1u;
            }
        }
    } else if (warp >= kScaleWarp) {   // scales
        const int r = threadIdx.x - 32 * kScaleWarp;
        const int blocks = p.K / 32;
        const int64_t row_bytes = scale_row_bytes(p.K), w_rows = (int64_t)p.E * mats * p.N;
        const int second = kGated ? p.N : kRowTile;
        // the next four steps' bytes are loaded while these four are stored
        long long ahead = blockIdx.x;
        int ahead_k = 0;
        Tile t = tile_at(p, tables, features, kFeatures, ahead);
        auto load = [&](uint32_t (&v)[4][8]) {
            if (ahead >= total)
                return;
            const int b0 = ahead_k * 8;
            int64_t w_row = (int64_t)t.expert * mats * p.N + t.feature + r;
            if (kMixed && r >= kRowTile / 2)
                w_row += p.N - kRowTile / 2;
            const int64_t row[4] = {w_row, w_row + second, (int64_t)t.row + r, (int64_t)t.row + r + 128};
            const bool in[4] = {w_row < w_rows, kTiles == 2 && w_row + second < w_rows, r < t.rows, r + 128 < t.rows};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (in[q])
                    scales32(v[q], q < 2 ? p.w_scales : p.scales, row[q], row_bytes, b0, blocks, q < 2 ? p.w_align : p.align);
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[q][i] = 0u;
            }
            ahead_k += 4;
            if (ahead_k >= steps) {
                ahead_k = 0;
                ahead += gridDim.x;
                if (ahead < total)
                    t = tile_at(p, tables, features, kFeatures, ahead);
            }
        };
        uint32_t now[4][8] = {}, next[4][8] = {};
        load(next);
        int stage = 0;
        uint32_t parity = 1u, buffer = 0u;
        // An atom is 128 rows by 4 blocks: row q's bytes are word q / 32 of 16-byte line q % 32, and in
        // tensor memory column q / 32 of lane q % 32, in each of the four lane quarters.  Atoms in
        // order: weights [tile][half of the step], tokens [half][group of 128 rows].
        constexpr uint32_t kTokenAtoms = kTiles * 1024;   // where the tokens' atoms begin
        const uint32_t buffers = mrr::smem_addr(smem) + p.sm_scales, buffer_size = kTokenAtoms + 1024 * groups;
        const uint32_t to = (r % 32) * 16 + (r / 32) * 4;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp % 4)) << 16) + p.sums * sums_columns;
        bool ok = true;
        for (long long i = blockIdx.x; ok && i < total; i += gridDim.x) {
            for (int k = 0; ok && k < steps; k += 4) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        now[q][j] = next[q][j];
                load(next);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (k + u >= steps)
                        break;
                    const uint32_t at = buffers + buffer * buffer_size;
                    buffer ^= 1u;
                    auto put = [&](uint32_t a, uint32_t v) {
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + a + to), "r"(v) : "memory");
                    };
                    put(0, now[0][2 * u]);
                    put(512, now[0][2 * u + 1]);
                    if (kTiles == 2) {
                        put(1024, now[1][2 * u]);
                        put(1536, now[1][2 * u + 1]);
                    }
                    put(kTokenAtoms, now[2][2 * u]);
                    put(kTokenAtoms + 512 * groups, now[2][2 * u + 1]);
                    if (groups == 2) {
                        put(kTokenAtoms + 512, now[3][2 * u]);
                        put(kTokenAtoms + 1536, now[3][2 * u + 1]);
                    }
                    // the other buffer is free again once all four warps are here
                    if (any_of(1, 128, !wait(p, sh, &sh->empty[stage], parity))) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t columns = lanes + stage * scale_columns;
#pragma unroll
                    for (int a = 0; a < 8; ++a)
                        if (a < 2 * kTiles + 2 * groups) {
                            uint32_t v[4];
                            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                                         : "r"(at + a * 512 + lane * 16)
                                         : "memory");
                            tc::store4(columns + 4 * a, v);
                        }
                    tc::store_wait();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0)
                        tc::mbar_arrive(mrr::smem_addr(&sh->full[stage]));
                    next_stage(stage, parity);
                }
            }
        }
    } else if (warp >= kEpilogueWarp) {
        const int quarter = warp % 4, part = (warp - kEpilogueWarp) / 4;   // lanes; every other 16 columns
        float *turn = reinterpret_cast<float *>(smem + p.sm_turn) + (warp - kEpilogueWarp) * 16 * kTurnPitch;
        int set = 0;
        uint32_t parity = 0u;
        for (long long i = blockIdx.x; i < total; i += gridDim.x) {
            const Tile t = tile_at(p, tables, features, kFeatures, i);
            const bool failed = !wait(p, sh, &sh->sums_full[set], parity);
            // kMixed: lane quarters 0 and 1 hold gate values, 2 and 3 the up values of the same features,
            // which change hands through shared memory; the two warps leave together
            const int pair = 2 + 2 * part + quarter % 2;
            if (kMixed ? any_of(pair, 64, failed) : failed)
                break;
            tc::fence_after();
            const int n0 = t.feature + 32 * (kMixed ? quarter % 2 : quarter);
            const uint32_t d = tmem + set * sums_columns + ((uint32_t)(32 * quarter) << 16);
            float *ups = reinterpret_cast<float *>(smem + p.sm_scales + 2 * (kTiles * 1024 + 1024 * groups)) +
                         (2 * part + quarter % 2) * 512 + lane;
            auto release = [&]() {   // the sums have been read
                tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(mrr::smem_addr(&sh->sums_empty[set]));
            };
            // the results of columns c .. c + 15, z those of the second tile
            auto results = [&](int c, int rows, float (&y)[16], float (&z)[16]) {
                uint32_t a[16], b[16];
                tc::load16(d + c, a);
                if (kTiles == 2)
                    tc::load16(d + p.tokens + c, b);
                tc::load_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    y[j] = __uint_as_float(a[j]);
                    if (kTiles == 2)
                        z[j] = __uint_as_float(b[j]);
                }
                if (kMixed) {
                    if (quarter >= 2)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            ups[32 * j] = y[j];
                    any_of(pair, 64, false);
                    if (quarter < 2)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            z[j] = ups[32 * j];
                    any_of(pair, 64, false);   // read: the next columns may come
                }
                if (kGated)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        y[j] = swiglu<kOut>(y[j], z[j]);
                if (p.row_weight) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float w = j < rows ? __ldg(p.row_weight + t.row + c + j) : 0.f;
                        y[j] *= w;
                        z[j] *= w;
                    }
                }
            };
            for (int c = 16 * part; c < t.columns; c += 32) {
                const int rows = min(16, t.rows - c);
                float y[16], z[16];
                results(c, rows, y, z);
                if (!kMixed || quarter < 2)
                    store16<kOut>(p, t.row + c, rows, n0, lane, turn, y);
                if (!kGated && kTiles == 2)
                    store16<kOut>(p, t.row + c, rows, n0 + kRowTile, lane, turn, z);
            }
            release();
            if (++set == p.sums) {
                set = 0;
                parity ^= 1u;
            }
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (sh->abort) {   // given up, by any warp: nothing may be in flight when the block leaves
        if (threadIdx.x == 0) {
            atomicOr(p.status, mrr_ws::kFlagTimeout);
            // a stage's copies have a moment to land; at most one of the two phases is not over
            for (int s = 0; s < p.stages; ++s)
                for (int b = 0; b < 2; ++b)
                    mrr::mbar_wait_bounded(mrr::smem_addr(&sh->full[s]), b, 1000000ull);
        }
        __syncwarp();
        if (warp == 1) {   // tensor memory is freed only after what was issued, by this thread, is done
            if (tc::elect()) {
                tc::commit(mrr::smem_addr(&sh->drained));
                mrr::mbar_wait_bounded(mrr::smem_addr(&sh->drained), 0, 100000000ull);
            }
            __syncwarp();
        }
    }
    if (warp == 1)
        tc::dealloc(tmem, kColumns);
}

template <bool kGated, int kOut, int kTiles>
cudaError_t launch_tiles(const Params &p, const Maps &maps, const mrr_device::Info &info, size_t smem,
                   cudaStream_t s)
{
    static std::atomic<uint64_t> allowed;
    auto kernel = grouped_kernel<kGated, kOut, kTiles>;
    const cudaError_t err = mrr_device::allow_smem(kernel, info, allowed);
    if (err != cudaSuccess)
        return err;
    kernel<<<info.sms, kThreads, smem, s>>>(p, maps);
    return cudaGetLastError();
}

template <bool kGated, int kOut>
cudaError_t launch(const Params &p, int tiles, const Maps &maps, const mrr_device::Info &info, size_t smem, cudaStream_t s)
{
    return tiles == 2 ? launch_tiles<kGated, kOut, 2>(p, maps, info, smem, s)
                      : launch_tiles<kGated, kOut, 1>(p, maps, info, smem, s);
}

}  // namespace

extern "C" {

size_t moe_mx_grouped_workspace(int64_t E) { return E < 1 ? 0 : mrr_ws::kHeaderBytes; }

// moe_mx_grouped_run with another limit on its waits, and short of an arrival on one kind of barrier (a
// Barrier): what a test calls to see a wait run out.  Not part of the library's interface.
mrr_status moe_mx_grouped_run_waits(const uint8_t *codes, const uint8_t *scales, int64_t A, int64_t K,
                                    const void *expert_num, int expert_num_is_i64, int64_t expert_num_type, int64_t E,
                                    const uint8_t *w_codes, const uint8_t *w_scales, int64_t N, int gated,
                                    const float *row_weight, void *out, moe_dtype out_dt, uint8_t *out_scales,
                                    void *workspace, size_t workspace_bytes, mrr_stream_t stream, uint64_t wait_ns,
                                    int short_of)
{
    if (out_dt != MOE_F16 && out_dt != MOE_BF16 && out_dt != MOE_F32 && out_dt != MOE_MXFP4)
        return MRR_ERR_DTYPE;
    if (expert_num_is_i64 != 0 && expert_num_is_i64 != 1)
        return MRR_ERR_DTYPE;
    if ((expert_num_type != 0 && expert_num_type != 1) || (gated != 0 && gated != 1))
        return MRR_ERR_ATTR;
    if (A < 0 || A > INT32_MAX - 256 || E < 1 || E > kMaxExperts || K < 32 || K % 32 || K > (1 << 20) || N < 1 ||
        N > (1 << 20) || E * N * (gated ? 2 : 1) > INT32_MAX - 512 || (out_dt == MOE_MXFP4 && N % 32))
        return MRR_ERR_SHAPE;
    if (!expert_num || !w_codes || !w_scales || (A > 0 && (!codes || !scales || !out)) ||
        (out_dt == MOE_MXFP4 && A > 0 && !out_scales))
        return MRR_ERR_NULL;
    const size_t out_size = out_dt == MOE_F32 ? 4 : (out_dt == MOE_MXFP4 ? 1 : 2);
    if ((uintptr_t)codes % 16 || (uintptr_t)w_codes % 16 || (uintptr_t)scales % 2 || (uintptr_t)w_scales % 2 ||
        (uintptr_t)expert_num % (expert_num_is_i64 ? 8 : 4) || (uintptr_t)row_weight % 4 || (uintptr_t)out % out_size)
        return MRR_ERR_ALIGN;
    if (!workspace || (uintptr_t)workspace % 256 || workspace_bytes < moe_mx_grouped_workspace(E))
        return MRR_ERR_WORKSPACE;
    mrr_device::Info info;
    if (!mrr_device::current(info)) {
        (void)cudaGetLastError();
        return MRR_ERR_CUDA;
    }
    Params p{};
    p.wait_ns = wait_ns, p.short_of = short_of;
    p.scales = scales, p.w_scales = w_scales;
    p.A = (int)A, p.K = (int)K, p.E = (int)E, p.N = (int)N;
    p.counts_i64 = expert_num_is_i64, p.counts_prefix = expert_num_type == 0, p.gated = gated, p.out_dt = (int)out_dt;
    p.counts = expert_num, p.row_weight = row_weight, p.out = out, p.out_scales = out_scales;
    p.status = static_cast<uint32_t *>(workspace);
    // Tiles of 256 weight rows by up to 192 token rows re-read either operand least, and fill tensor
    // memory beside the scales.  Tiles of 128 weight rows cost more than half as much each, but there are
    // twice as many: taken where that fills the last round of blocks so much better that it pays.
    // rounds() estimates how many tiles a block gets (the counts are on the device): an expert with
    // rows has one token tile up to 96 rows on average, then half a tile more than its rows fill.
    //  * Up to 24 rows an expert a tile's time is its weights', half of it for 128 rows.  32 experts of
    //    7168 x 2048, gated, 512 rows: 83 us (7 rounds) against 86 (4); 16 experts, 385 rows: 51 (4)
    //    against 45 (2).  Tiles of 64 token rows then leave room for more stages and two sets of sums,
    //    so that a tile's results are written under the next one: 82.8 us against 85.5 with 192.
    //  * Above, 128 weight rows cost some two thirds of 256.  8 experts of 7168 x 1024, gated, 1024
    //    rows: 22 us (1 round) against 25 (1); 1536 rows: 35 (2) against 27 (1).
    const int mats = gated ? 2 : 1;
    const bool few = A <= kFewRows * E;
    const int64_t token_tiles = A <= 96 * E ? (A < E ? A : E) : A / 192 + E / 2;
    auto rounds = [&](int rows) { return ((N * mats + rows - 1) / rows * token_tiles + info.sms - 1) / info.sms; };
    const int tiles = few ? (rounds(kRowTile) < 2 * rounds(2 * kRowTile) ? 1 : 2)
                          : (2 * rounds(kRowTile) < 3 * rounds(2 * kRowTile) ? 1 : 2);
    p.tokens = few && tiles == 1 ? 64 : 192;
    p.sums = p.tokens <= 64 ? 2 : 1;
    auto aligned = [K](const void *s) {
        const uint64_t both = (uintptr_t)s | (uint64_t)scale_row_bytes(K);
        return both % 32 == 0 ? 32 : both % 16 == 0 ? 16 : both % 8 == 0 ? 8 : 2;
    };
    p.align = aligned(scales);
    p.w_align = aligned(w_scales);
    if (out_dt == MOE_MXFP4)
        p.out_wide = (uintptr_t)out % 8 == 0 ? 8 : 0;
    else
        p.out_wide = (uintptr_t)out % 32 == 0 && N % 16 == 0 ? 32 : (uintptr_t)out % 8 == 0 && N % 4 == 0 ? 8 : 0;
    p.sm_tables = (int)mrr_ws::round_up(sizeof(Shared), 16);
    p.sm_scales = (int)mrr_ws::round_up(p.sm_tables + 8 * (E + 1), 16);
    p.sm_turn = p.sm_scales + 2 * (tiles * 1024 + 1024 * groups_of(p.tokens)) + (gated && tiles == 1 ? 4 * 2048 : 0);
    p.sm_stage = (int)mrr_ws::round_up(
        p.sm_turn + (out_dt != MOE_F32 ? kEpilogueWarps * 16 * kTurnPitch * 4 : 0), 1024);
    const int columns_left = (kColumns - p.sums * tiles * p.tokens) / (8 * tiles + 8 * groups_of(p.tokens));
    int stages = (info.smem_max - p.sm_stage) / stage_bytes(tiles, p.tokens);
    stages = stages < columns_left ? stages : columns_left;
    p.stages = stages < kMaxStages ? stages : kMaxStages;
    if (p.stages < 2)
        return MRR_ERR_CUDA;
    Maps maps;
    bool made = tc::make_map(&maps.w, w_codes, E * N * (gated ? 2 : 1), K / 2,
                             gated && tiles == 1 ? kRowTile / 2 : kRowTile);
    for (int i = 0; i < 4; ++i)
        made = made && tc::make_map(&maps.x[i], A ? codes : w_codes, A ? A : 1, K / 2, box_rows(i));
    if (!made)
        return MRR_ERR_CUDA;
    const size_t smem = (size_t)p.sm_stage + (size_t)p.stages * stage_bytes(tiles, p.tokens);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err;
    if (out_dt == MOE_BF16)
        err = gated ? launch<true, MOE_BF16>(p, tiles, maps, info, smem, st) : launch<false, MOE_BF16>(p, tiles, maps, info, smem, st);
    else if (out_dt == MOE_F16)
        err = gated ? launch<true, MOE_F16>(p, tiles, maps, info, smem, st) : launch<false, MOE_F16>(p, tiles, maps, info, smem, st);
    else if (out_dt == MOE_F32)
        err = gated ? launch<true, MOE_F32>(p, tiles, maps, info, smem, st) : launch<false, MOE_F32>(p, tiles, maps, info, smem, st);
    else
        err = gated ? launch<true, MOE_MXFP4>(p, tiles, maps, info, smem, st) : launch<false, MOE_MXFP4>(p, tiles, maps, info, smem, st);
    if (err != cudaSuccess) {
        (void)cudaGetLastError();
        return MRR_ERR_CUDA;
    }
    return MRR_OK;
}

mrr_status moe_mx_grouped_run(const uint8_t *codes, const uint8_t *scales, int64_t A, int64_t K,
                              const void *expert_num, int expert_num_is_i64, int64_t expert_num_type, int64_t E,
                              const uint8_t *w_codes, const uint8_t *w_scales, int64_t N, int gated,
                              const float *row_weight, void *out, moe_dtype out_dt, uint8_t *out_scales,
                              void *workspace, size_t workspace_bytes, mrr_stream_t stream)
{
    return moe_mx_grouped_run_waits(codes, scales, A, K, expert_num, expert_num_is_i64, expert_num_type, E, w_codes,
                                    w_scales, N, gated, row_weight, out, out_dt, out_scales, workspace, workspace_bytes,
                                    stream, kWaitLimitNs, kNone);
}

}  // extern "C"
