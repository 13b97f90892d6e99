// Tokens laid out by expert (include/moe_tokens.h): a stable counting sort of the slots by expert,
// and the move of every token's row to its k places.
//
// A slot's row is the number of slots whose (key, slot) is smaller, slots without an expert here
// having the key E behind all others: their rows are the rows of zeros.  The threads that have a
// token read it once and write it to its k places: T (1 + k) rows of traffic, the least there is.
// HBM bounds it.
//
// Few slots (sort_few, up to 4096): one launch.  Each block looks at all keys and counts the smaller ones for its own
// slots only.  More (sort_index, up to 131072): one cluster ranks them all, each warp a share that it holds in registers, the
// counts passed round through shared memory; a second launch moves the rows.  More slots or experts still: a first launch of
// one cluster counts the keys of kChunks chunks and leaves where each chunk's slots of each key begin (sort_count); in the
// second each block ranks its own slots, having counted those of its chunk ahead of them while the first ran (sort_rank);
// the third moves the rows.  600 tokens of 2048 to 8 experts: 12.6 us with sort_index, 19 with the three launches; 16384 of
// 7168: 333 and 332.
//
// The move has many small blocks that take the tokens in order, so that what is written at a time lies close together: with
// blocks that stay and rank and move a share of the tokens each, 16384 x 7168 bfloat16 to 8 experts took 355 us.  Its rows
// take 313 us of the 329, 6.8 TB/s.
#include <atomic>
#include <string.h>

#include "device_info.h"
#include "moe_tokens.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
using moe_rows::kFull;
constexpr uint32_t kNone = 0x80000000u;   // beside a row: the slot has no expert here, the row is zeros
constexpr int kMoveThreads = 256;         // most threads of a block of sort_move
constexpr int kMoveAtOnce = 4;            // vectors of a row that one of them has under way
constexpr int kZeroBlocks = 2432;         // behind the tokens' blocks, sixteen for each of the 152 SMs
constexpr int kAnyThreads = 128;          // of sort_move_any
constexpr int kAnySegment = 8192;         // bytes of a row that it has in shared memory
constexpr int kFewSlots = 4096;
constexpr int kFewMine = 128;             // most slots of a block of sort_few
constexpr int kBatch = 1024;              // slots that a block of sort_rank ranks at once
constexpr int kMaxE = MOE_SORT_MAX_EXPERTS;
constexpr int kGroups = 608;              // blocks of sort_rank: four on each of the 152 SMs
constexpr int kCluster = 16;              // blocks of sort_count
constexpr int kCountThreads = 1024;
constexpr int kOfBlock = 4;               // chunks of one of them
constexpr int kChunks = kCluster * kOfBlock;
constexpr int kRounds = 8;                // slots of a thread of sort_index
constexpr int kIndexSlots = kCluster * kCountThreads * kRounds;
constexpr int kIndexE = 1023;             // its most experts: a thread has a key

struct Params {
    const void *idx;
    uint64_t first;
    const uint8_t *x, *scales;
    const void *weight;
    uint8_t *out, *out_scales;
    float *out_weight;
    int32_t *token_idx, *row_idx;
    void *num;
    uint32_t *table;
    int64_t row_bytes, row_stride, scale_row_bytes;
    int64_t T;
    uint32_t n;        // T * k
    int k, E;
    int idx64, weight_dt, cumsum, scale_unit;
    int tokens;        // a block's tokens (the last block's: fewer)
    int groups;        // blocks along the tokens
    int parts;         // the table: chunks of `parts` blocks' slots, kChunks at most
    int group, move_tokens;   // the move: threads of a token, tokens of a block
};

__device__ __forceinline__ uint32_t key_of(const Params &p, uint32_t slot)
{
    const uint64_t v = p.idx64 ? (uint64_t)__ldg(static_cast<const long long *>(p.idx) + slot)
                               : (uint64_t)(int64_t)__ldg(static_cast<const int *>(p.idx) + slot);
    const uint64_t d = v - p.first;   // unsigned: anything below `first` is far above E
    return d < (uint64_t)p.E ? (uint32_t)d : (uint32_t)p.E;
}

// f(slot, key) of slots lo .. hi - 1, by threads 0 .. THREADS - 1: eight loads a thread under way at once
template <int THREADS, typename F>
__device__ __forceinline__ void keys_of(const Params &p, uint32_t lo, uint32_t hi, uint32_t thread, F f)
{
    for (uint32_t i = lo + thread; i < hi; i += 8 * THREADS) {
        uint32_t key[8];
#pragma unroll
        for (uint32_t u = 0; u < 8; ++u)
            key[u] = i + u * THREADS < hi ? key_of(p, i + u * THREADS) : 0u;
#pragma unroll
        for (uint32_t u = 0; u < 8; ++u)
            if (i + u * THREADS < hi)
                f(i + u * THREADS, key[u]);
    }
}

template <int W>
struct Vec;
template <>
struct Vec<16> { using T = uint4; };
template <>
struct Vec<8> { using T = uint2; };
template <>
struct Vec<4> { using T = uint32_t; };
template <>
struct Vec<2> { using T = uint16_t; };
template <>
struct Vec<1> { using T = uint8_t; };

// shared memory of a token of sort_move_any: a segment that begins anywhere in 16 bytes, and a word of 16 behind it
__host__ __device__ __forceinline__ int any_space(int64_t row_bytes)
{
    return (int)((row_bytes < kAnySegment ? row_bytes : kAnySegment) + 15) / 16 * 16 + 32;
}

template <typename V>
__device__ __forceinline__ V zero_of()
{
    V v;
    memset(&v, 0, sizeof(v));
    return v;
}

// Move tokens first .. first + count - 1 (their slots' rows in `rows`, k for each) : vectors v0 .. v1 - 1 of
// W bytes of each.  A warp takes kEach vectors a lane of one token, all loaded before the first is stored.
template <int W>
__device__ __forceinline__ void move_rows(const Params &p, int64_t first, int count, const uint32_t *rows, int v0, int v1)
{
    using V = typename Vec<W>::T;
    constexpr int kEach = 4;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int segs = (v1 - v0 + 32 * kEach - 1) / (32 * kEach);
    for (int u = warp; u < count * segs; u += kWarps) {
        const int t = u / segs, at = v0 + (u - t * segs) * 32 * kEach + lane;
        const uint32_t *r = rows + t * p.k;
        bool any = false;
        for (int j = 0; j < p.k; ++j)
            any |= !(r[j] & kNone);
        V v[kEach];
        const V *from = reinterpret_cast<const V *>(p.x + (first + t) * p.row_stride);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            v[i] = any && at + 32 * i < v1 ? __ldg(from + at + 32 * i) : zero_of<V>();
        for (int j = 0; j < p.k; ++j) {
            const uint32_t row = r[j];
            V *to = reinterpret_cast<V *>(p.out + (int64_t)(row & ~kNone) * p.row_bytes);
            if (row & kNone) {
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (at + 32 * i < v1)
                        to[at + 32 * i] = zero_of<V>();
            } else {
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (at + 32 * i < v1)
                        to[at + 32 * i] = v[i];
            }
        }
    }
}

__device__ __forceinline__ float weight_of(const Params &p, int64_t slot)
{
    return p.weight_dt == MOE_F32    ? moe_mx::load1<MOE_F32>(p.weight, slot)
           : p.weight_dt == MOE_BF16 ? moe_mx::load1<MOE_BF16>(p.weight, slot)
                                     : moe_mx::load1<MOE_F16>(p.weight, slot);
}

// The slots first .. first + count - 1: their index entries and weights.
__device__ __forceinline__ void write_slots(const Params &p, uint32_t first, int count, const uint32_t *rows)
{
    for (int s = threadIdx.x; s < count; s += kThreads) {
        const uint32_t slot = first + s, row = rows[s] & ~kNone;
        const bool none = rows[s] & kNone;
        p.row_idx[slot] = none ? -1 : (int32_t)row;
        p.token_idx[row] = none ? -1 : (int32_t)slot;
        if (p.out_weight) {
            p.out_weight[row] = none ? 0.0f : weight_of(p, slot);
        }
    }
}

// Their scales, in 4-byte units where rows and both pointers allow it, else bytes.
__device__ __forceinline__ void write_scales(const Params &p, uint32_t first, int count, const uint32_t *rows)
{
    if (!p.out_scales)
        return;
    const int64_t units = p.scale_row_bytes / p.scale_unit;
    for (int64_t i = threadIdx.x; i < count * units; i += kThreads) {
        const int64_t s = i / units, at = i - s * units;
        const uint32_t row = rows[s];
        const int64_t from = (int64_t)((first + (uint32_t)s) / (uint32_t)p.k) * units + at;
        const int64_t to = (int64_t)(row & ~kNone) * units + at;
        if (p.scale_unit == 4)
            reinterpret_cast<uint32_t *>(p.out_scales)[to] =
                row & kNone ? 0u : __ldg(reinterpret_cast<const uint32_t *>(p.scales) + from);
        else
            p.out_scales[to] = row & kNone ? (uint8_t)0 : __ldg(p.scales + from);
    }
}

__device__ __forceinline__ void store_num(const Params &p, int e, uint32_t v)
{
    if (p.idx64)
        static_cast<long long *>(p.num)[e] = v;
    else
        static_cast<int *>(p.num)[e] = (int)v;
}

// v[0 .. count - 1] to its exclusive prefix, by a block of THREADS threads
template <int THREADS>
__device__ __forceinline__ void block_prefix(uint32_t *v, int count)
{
    __shared__ uint32_t of_warp[THREADS / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int per = (count + THREADS - 1) / THREADS, lo = threadIdx.x * per, hi = min(count, lo + per);
    uint32_t sum = 0;
    for (int i = lo; i < hi; ++i)
        sum += v[i];
    uint32_t upto = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t o = __shfl_up_sync(kFull, upto, d);
        upto += lane >= d ? o : 0u;
    }
    if (lane == 31)
        of_warp[warp] = upto;
    __syncthreads();
    uint32_t at = upto - sum;
    for (int w = 0; w < warp; ++w)
        at += of_warp[w];
    for (int i = lo; i < hi; ++i) {
        const uint32_t c = v[i];
        v[i] = at;
        at += c;
    }
    __syncthreads();
}

// The share of the row's vectors that this block's y index has.
__device__ __forceinline__ void my_vectors(int vectors, int &v0, int &v1)
{
    const int per = (vectors + gridDim.y - 1) / gridDim.y;
    v0 = min(vectors, (int)blockIdx.y * per);
    v1 = min(vectors, v0 + per);
}

template <int W>
__global__ void __launch_bounds__(kThreads) sort_few(Params p)
{
    // (key, slot) as one number: 13 bits over 12
    __shared__ __align__(16) uint32_t order[kFewSlots];
    __shared__ uint32_t rows[kFewMine];
    if (blockIdx.x == (unsigned)p.groups) {   // one more block: the experts' counts
        if (blockIdx.y != 0)
            return;
        for (int e = threadIdx.x; e < p.E; e += kThreads)
            order[e] = 0u;
        __syncthreads();
        keys_of<kThreads>(p, 0, p.n, threadIdx.x, [&](uint32_t, uint32_t key) {
            if (key < (uint32_t)p.E)
                atomicAdd(&order[key], 1u);
        });
        __syncthreads();
        if (!p.cumsum) {
            for (int e = threadIdx.x; e < p.E; e += kThreads)
                store_num(p, e, order[e]);
        } else {
            // an expert's inclusive prefix is its exclusive one and its count
            uint32_t own[kMaxE / kThreads];
            for (int e = threadIdx.x, i = 0; e < p.E; e += kThreads, ++i)
                own[i] = order[e];
            __syncthreads();
            block_prefix<kThreads>(order, p.E);
            for (int e = threadIdx.x, i = 0; e < p.E; e += kThreads, ++i)
                store_num(p, e, order[e] + own[i]);
        }
        return;
    }
    const uint32_t n4 = (p.n + 3) / 4 * 4;
    keys_of<kThreads>(p, 0, p.n, threadIdx.x, [&](uint32_t i, uint32_t key) { order[i] = key << 12 | i; });
    if (threadIdx.x < n4 - p.n)
        order[p.n + threadIdx.x] = 0xffffffffu;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
    const int tokens = (int)min((int64_t)p.tokens, p.T - t0), mine = tokens * p.k;
    const uint32_t s0 = (uint32_t)t0 * p.k;
    const int lane = threadIdx.x % 32;
    for (int s = threadIdx.x / 32; s < mine; s += kWarps) {
        const uint32_t own = order[s0 + s];
        uint32_t smaller = 0;
        for (uint32_t i = 4 * lane; i < n4; i += 128) {
            const uint4 o = *reinterpret_cast<const uint4 *>(order + i);
            smaller += (o.x < own) + (o.y < own) + (o.z < own) + (o.w < own);
        }
        smaller = __reduce_add_sync(kFull, smaller);
        if (lane == 0)
            rows[s] = smaller | (own >> 12 == (uint32_t)p.E ? kNone : 0u);
    }
    __syncthreads();
    if (blockIdx.y == 0) {
        write_slots(p, s0, mine, rows);
        write_scales(p, s0, mine, rows);
    }
    if (p.out) {
        int v0, v1;
        my_vectors((int)(p.row_bytes / W), v0, v1);
        move_rows<W>(p, t0, tokens, rows, v0, v1);
    }
}

// behind the table: the number of rows that experts have
__device__ __forceinline__ uint32_t *used_rows(const Params &p) { return p.table + kChunks * (p.E + 1); }

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// the word at shared-memory address `at` of block `rank` of the cluster
__device__ __forceinline__ uint32_t load_from_block(uint32_t at, uint32_t rank)
{
    uint32_t there, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(there) : "memory");
    return v;
}

// table[c][e] = the row of chunk c's first slot of key e (E: none).  One cluster; a block has kOfBlock chunks.
// Shared memory: all[E + 1], and count[kOfBlock][E + 1].
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kCountThreads) sort_count(Params p)
{
    mrr::grid_launch_dependents();
    extern __shared__ uint32_t all[];
    const int keys = p.E + 1;
    uint32_t *count = all + keys;
    for (int e = threadIdx.x; e < kOfBlock * keys; e += kCountThreads)
        count[e] = 0u;
    __syncthreads();
    {
        constexpr int kEach = kCountThreads / kOfBlock;
        const int mine = threadIdx.x / kEach;
        const uint64_t chunk = blockIdx.x * kOfBlock + mine, per = (uint64_t)p.parts * p.tokens * p.k;
        keys_of<kEach>(p, (uint32_t)min((uint64_t)p.n, chunk * per), (uint32_t)min((uint64_t)p.n, (chunk + 1) * per),
                       threadIdx.x % kEach, [&](uint32_t, uint32_t key) { atomicAdd(&count[mine * keys + key], 1u); });
    }
    __syncthreads();
    // a key's counts to what its chunks ahead, in this block, have; and the block's own
    for (int e = threadIdx.x; e < keys; e += kCountThreads) {
        uint32_t sum = 0;
#pragma unroll
        for (int c = 0; c < kOfBlock; ++c) {
            const uint32_t v = count[c * keys + e];
            count[c * keys + e] = sum;
            sum += v;
        }
        all[e] = sum;
    }
    cluster_barrier();
    uint32_t sum[(kMaxE + kCountThreads) / kCountThreads];
    const uint32_t from = mrr::smem_addr(all);
    int turn = 0;
    for (int e = threadIdx.x; e < keys; e += kCountThreads, ++turn) {
        uint32_t total = 0, ahead = 0;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) {
            const uint32_t v = load_from_block(from + 4 * e, r);
            total += v;
            ahead += r < (int)blockIdx.x ? v : 0u;
        }
        sum[turn] = total;
#pragma unroll
        for (int c = 0; c < kOfBlock; ++c)
            count[c * keys + e] += ahead;
    }
    cluster_barrier();   // all[] is read no more
    turn = 0;
    for (int e = threadIdx.x; e < keys; e += kCountThreads, ++turn)
        all[e] = sum[turn];
    __syncthreads();
    block_prefix<kCountThreads>(all, keys);
    turn = 0;
    for (int e = threadIdx.x; e < keys; e += kCountThreads, ++turn) {
        const uint32_t first = all[e];
#pragma unroll
        for (int c = 0; c < kOfBlock; ++c)
            p.table[(size_t)(blockIdx.x * kOfBlock + c) * keys + e] = first + count[c * keys + e];
        if (blockIdx.x == 0 && e < p.E)
            store_num(p, e, p.cumsum ? first + sum[turn] : sum[turn]);
        if (blockIdx.x == 0 && e == p.E)
            *used_rows(p) = first;
    }
}

// The counts of the keys (all[e] of each block of the cluster) to where this block's slots of key e begin, in all[e] too;
// the experts' numbers and the rows they have are written by the first block.  A thread has a key (keys <= its threads).
__device__ __forceinline__ void begin_of_keys(const Params &p, uint32_t *all, int keys)
{
    cluster_barrier();
    const uint32_t from = mrr::smem_addr(all);
    const int e = threadIdx.x;
    uint32_t total = 0, ahead = 0;
    if (e < keys) {
#pragma unroll
        for (int r = 0; r < kCluster; ++r) {
            const uint32_t v = load_from_block(from + 4 * e, r);
            total += v;
            ahead += r < (int)blockIdx.x ? v : 0u;
        }
    }
    cluster_barrier();   // all[] is read no more
    if (e < keys)
        all[e] = total;
    __syncthreads();
    block_prefix<kCountThreads>(all, keys);
    if (e < keys) {
        const uint32_t first = all[e];
        if (blockIdx.x == 0 && e < p.E)
            store_num(p, e, p.cumsum ? first + total : total);
        if (blockIdx.x == 0 && e == p.E)
            *used_rows(p) = first;
        all[e] = first + ahead;
    }
    __syncthreads();
}

// Every slot's row, for up to kIndexSlots slots.  One cluster; a warp has 32 slots at a time, p.parts times, in order.
// Shared memory: all[E + 1], and count[warps][E + 1] of 16 bits.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kCountThreads) sort_index(Params p)
{
    mrr::grid_launch_dependents();
    extern __shared__ uint32_t all[];
    const int keys = p.E + 1, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint16_t *counts = reinterpret_cast<uint16_t *>(all + keys), *mine = counts + warp * keys;
    const uint32_t s0 = (blockIdx.x * (kCountThreads / 32) + warp) * 32 * p.parts + lane;
    uint32_t slot[kRounds];   // key << 16 | the number of this warp's slots of the key ahead of it
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
        slot[r] = r < p.parts && s0 + 32 * r < p.n ? key_of(p, s0 + 32 * r) : keys;
    for (int e = lane; e < keys; e += 32)
        mine[e] = 0;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        if (r >= p.parts)
            break;
        const uint32_t key = slot[r], same = __match_any_sync(kFull, key);
        const uint32_t at = key < (uint32_t)keys ? mine[key] : 0u;
        __syncwarp();
        slot[r] = key << 16 | (at + __popc(same & ((1u << lane) - 1)));
        if (key < (uint32_t)keys && lane == __ffs(same) - 1)
            mine[key] = (uint16_t)(at + __popc(same));
        __syncwarp();
    }
    __syncthreads();
    // each warp's counts to what the warps ahead of it, in this block, have
    if (threadIdx.x < keys) {
        uint32_t sum = 0;
#pragma unroll 8
        for (int w = 0; w < kCountThreads / 32; ++w) {
            const uint32_t v = counts[w * keys + threadIdx.x];
            counts[w * keys + threadIdx.x] = (uint16_t)sum;
            sum += v;
        }
        all[threadIdx.x] = sum;
    }
    begin_of_keys(p, all, keys);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint32_t key = slot[r] >> 16;
        if (r < p.parts && key < (uint32_t)keys)
            p.row_idx[s0 + 32 * r] = key == (uint32_t)p.E ? -1 : (int32_t)(all[key] + mine[key] + (slot[r] & 0xffffu));
    }
}

// Every slot's row.  Each block has p.tokens tokens.
__global__ void __launch_bounds__(kThreads) sort_rank(Params p)
{
    mrr::grid_launch_dependents();
    __shared__ uint32_t base[kMaxE + 2];   // of each key: the row of this block's next slot
    __shared__ uint32_t before[kMaxE + 1]; // of each key: its slots ahead of this block's
    __shared__ uint32_t rows[kBatch];
    const int lane = threadIdx.x % 32;
    const int chunk = blockIdx.x / p.parts;
    for (int e = threadIdx.x; e <= p.E; e += kThreads)
        before[e] = 0u;
    __syncthreads();
    // slots of this chunk ahead of this block's
    const uint64_t each = (uint64_t)p.tokens * p.k;
    keys_of<kThreads>(p, (uint32_t)(chunk * p.parts * each), (uint32_t)(blockIdx.x * each), threadIdx.x,
                      [&](uint32_t, uint32_t key) { atomicAdd(&before[key], 1u); });
    __syncthreads();
    mrr::grid_dependency_wait();   // the table is the previous launch's
    for (int e = threadIdx.x; e <= p.E; e += kThreads)
        base[e] = before[e] + p.table[(size_t)chunk * (p.E + 1) + e];

    const uint32_t s_end = (uint32_t)min((uint64_t)p.n, (blockIdx.x + 1) * each);
    for (uint32_t s0 = (uint32_t)(blockIdx.x * each); s0 < s_end; s0 += kBatch) {
        const int mine = (int)min((uint32_t)kBatch, s_end - s0);
        __syncthreads();   // the batch before has been written
        for (int s = threadIdx.x; s < mine; s += kThreads)
            rows[s] = key_of(p, s0 + s);
        __syncthreads();
        if (threadIdx.x < 32) {
            // 32 slots at a time, in order: slots of one key follow each other in lane order
            for (int s = lane; s < mine + lane; s += 32) {
                const uint32_t key = s < mine ? rows[s] : (uint32_t)p.E + 1;
                const uint32_t same = __match_any_sync(kFull, key);
                const uint32_t at = base[key];
                __syncwarp();
                if (s < mine)
                    rows[s] = (at + __popc(same & ((1u << lane) - 1))) | (key == (uint32_t)p.E ? kNone : 0u);
                if (lane == __ffs(same) - 1)
                    base[key] = at + __popc(same);
                __syncwarp();
            }
        }
        __syncthreads();
        for (int s = threadIdx.x; s < mine; s += kThreads)
            p.row_idx[s0 + s] = rows[s] & kNone ? -1 : (int32_t)rows[s];
    }
}

// What moves with a token's rows: their slots, weights and scale rows (in 4-byte units where rows and both pointers
// allow it, else bytes).
__device__ __forceinline__ void move_small(const Params &p, int64_t t, int lane)
{
    const int32_t *rows = p.row_idx + t * p.k;
    for (int j = lane; j < p.k; j += p.group) {
        const int32_t row = rows[j];
        if (row < 0)
            continue;
        p.token_idx[row] = (int32_t)(t * p.k) + j;
        if (p.out_weight)
            p.out_weight[row] = weight_of(p, t * p.k + j);
    }
    if (!p.out_scales)
        return;
    const int units = (int)(p.scale_row_bytes / p.scale_unit);
    for (int c = lane; c < units; c += p.group) {
        if (p.scale_unit == 4) {
            const uint32_t s = __ldg(reinterpret_cast<const uint32_t *>(p.scales) + t * units + c);
            for (int j = 0; j < p.k; ++j)
                if (rows[j] >= 0)
                    reinterpret_cast<uint32_t *>(p.out_scales)[(int64_t)rows[j] * units + c] = s;
        } else {
            const uint8_t s = __ldg(p.scales + t * units + c);
            for (int j = 0; j < p.k; ++j)
                if (rows[j] >= 0)
                    p.out_scales[(int64_t)rows[j] * units + c] = s;
        }
    }
}

// A block's share of the rows of zeros: every `blocks`th piece of 16 KB of them, so that what all blocks write at a
// time lies together (16384 x 7168 bfloat16 with an eighth of the experts held here: 328 us; 423 with one long piece for
// each of 608 blocks; 4099 x 2050 float16 with a third: 26 and 34).
__device__ __forceinline__ void clear_rest(const Params &p, int64_t block, int64_t blocks)
{
    const int64_t used = *used_rows(p);
    auto share = [&](uint8_t *out, int64_t row_bytes) {
        constexpr int64_t kPiece = 16384;
        const int64_t lo = used * row_bytes, all = p.n * row_bytes - lo;
        for (int64_t at = block * kPiece; at < all; at += blocks * kPiece)
            moe_rows::clear<1>(out, lo + at, min(kPiece, all - at), threadIdx.x, blockDim.x);
    };
    if (p.out)
        share(p.out, p.row_bytes);
    if (p.out_scales)
        share(p.out_scales, p.scale_row_bytes);
    for (int64_t r = used + block * blockDim.x + threadIdx.x; r < p.n; r += blocks * blockDim.x) {
        p.token_idx[r] = -1;
        if (p.out_weight)
            p.out_weight[r] = 0.0f;
    }
}

// The rows, of p.move_tokens tokens a block and a group of p.group threads to a token, and behind them blocks that
// write the rows of zeros.  kEach vectors of a row are loaded before the first is stored, the first ones before the
// ranks are there (x is no output of the launches before).
__global__ void __launch_bounds__(kMoveThreads) sort_move(Params p)
{
    constexpr int kEach = kMoveAtOnce;
    const int64_t token_blocks = (p.T + p.move_tokens - 1) / p.move_tokens;
    const int vectors = (int)(p.row_bytes / 16);
    if (blockIdx.x >= token_blocks) {
        mrr::grid_dependency_wait();
        clear_rest(p, blockIdx.x - token_blocks, gridDim.x - token_blocks);
        return;
    }
    const int of_block = threadIdx.x / p.group, lane = threadIdx.x - of_block * p.group;
    const int64_t t = (int64_t)blockIdx.x * p.move_tokens + of_block;
    if (t >= p.T)
        return;
    const uint4 *from = reinterpret_cast<const uint4 *>(p.x + t * p.row_stride);
    uint4 v[kEach];
    auto load = [&](int c) {
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (c + i * p.group < vectors)
                v[i] = __ldg(from + c + i * p.group);
    };
    load(lane);
    mrr::grid_dependency_wait();
    const int32_t *rows = p.row_idx + t * p.k;
    for (int c = lane; c < vectors;) {
        for (int j0 = 0; j0 < p.k; j0 += 8) {
            int32_t row[8];   // all loaded before the first store, which the compiler could not tell apart from them
#pragma unroll
            for (int j = 0; j < 8; ++j)
                row[j] = j0 + j < p.k ? rows[j0 + j] : -1;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (row[j] < 0)
                    continue;
                uint4 *to = reinterpret_cast<uint4 *>(p.out + row[j] * p.row_bytes);
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (c + i * p.group < vectors)
                        to[c + i * p.group] = v[i];
            }
        }
        c += kEach * p.group;
        load(c);
    }
    move_small(p, t, lane);
}

// `size` bytes that begin `ahead` bytes behind a 16-byte boundary, as whole words of 16 from `first` to `last` (counted from
// the boundary) and the bytes at both ends that share their 16 with something else.
struct Ends {
    int first, last, bytes, head, start;

    __device__ __forceinline__ Ends(int ahead, int size)
        : first((ahead + 15) & ~15), last((ahead + size) & ~15), start(ahead)
    {
        head = min(first - ahead, size);
        bytes = first > last ? size : head + ahead + size - last;
    }

    // the i-th of the bytes
    __device__ __forceinline__ int at(int i) const { return i < head ? start + i : last + i - head; }
};

// The same for rows of any size and alignment.  A segment of a token's row is brought to shared memory, placed as it lies
// towards 16-byte boundaries; for each place it goes to, a thread makes the aligned 16 bytes of the output out of two
// words of shared memory, by a shift that is the same for the whole row.  Bytes at the ends of a segment, that share
// their 16 with another's, are moved singly, a lane each.  (In pieces of the widest size that all rows are multiples of
// instead: 8192 x 2049 bfloat16 to 6 experts 66 us, this way 50; 8192 x 4097 int8 to 4 164 and 39.)
__global__ void __launch_bounds__(kAnyThreads) sort_move_any(Params p)
{
    extern __shared__ __align__(16) uint8_t space[];
    const int64_t token_blocks = (p.T + p.move_tokens - 1) / p.move_tokens;
    if (blockIdx.x >= token_blocks) {
        mrr::grid_dependency_wait();
        clear_rest(p, blockIdx.x - token_blocks, gridDim.x - token_blocks);
        return;
    }
    const int of_block = threadIdx.x / p.group, lane = threadIdx.x - of_block * p.group;
    const int64_t t = (int64_t)blockIdx.x * p.move_tokens + of_block;
    const bool mine = t < p.T;   // the whole block stays for its barriers
    const uint8_t *src = p.x + (mine ? t : 0) * p.row_stride;
    uint8_t *here = space + of_block * any_space(p.row_bytes);
    const int32_t *rows = p.row_idx + (mine ? t : 0) * p.k;
    for (int64_t at = 0; at < p.row_bytes; at += kAnySegment) {
        const int size = (int)min((int64_t)kAnySegment, p.row_bytes - at);
        const uint8_t *from = src + at;
        const int shift = (int)((uintptr_t)from % 16);   // where the segment begins in shared memory
        if (at)
            __syncthreads();   // the segment before has been read
        if (mine) {
            const Ends ends(shift, size);
            for (int c = ends.first + 16 * lane; c < ends.last; c += 16 * p.group)
                *reinterpret_cast<uint4 *>(here + c) = __ldg(reinterpret_cast<const uint4 *>(from - shift + c));
            for (int i = lane; i < ends.bytes; i += p.group)
                here[ends.at(i)] = __ldg(from - shift + ends.at(i));
        }
        __syncthreads();
        if (at == 0)
            mrr::grid_dependency_wait();
        if (!mine)
            continue;
        for (int j = 0; j < p.k; ++j) {
            const int32_t row = rows[j];
            if (row < 0)
                continue;
            uint8_t *to = p.out + row * p.row_bytes + at;
            const int ahead = (int)((uintptr_t)to % 16);   // of the segment, in its first 16 bytes
            const uint32_t m = (uint32_t)(shift - ahead) & 15u, bits = (m & 3u) * 8u;
            const Ends ends(ahead, size);
            for (int c = ends.first + 16 * lane; c < ends.last; c += 16 * p.group) {
                const uint4 *q = reinterpret_cast<const uint4 *>(here + (shift - ahead + c - (int)m));
                const uint4 a = q[0], b = q[1];
                uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                if (m & 8u) {
#pragma unroll
                    for (int i = 0; i < 6; ++i)
                        w[i] = w[i + 2];
                }
                if (m & 4u) {
#pragma unroll
                    for (int i = 0; i < 5; ++i)
                        w[i] = w[i + 1];
                }
                *reinterpret_cast<uint4 *>(to - ahead + c) =
                    make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                               __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
            }
            for (int i = lane; i < ends.bytes; i += p.group)
                (to - ahead)[ends.at(i)] = here[shift - ahead + ends.at(i)];
        }
    }
    if (mine)
        move_small(p, t, lane);
}

// How the work is cut, from the sizes alone.  A chunk is at most 10 of sort_rank's blocks.
void cut(int64_t T, int64_t &tokens, int64_t &groups, int64_t &parts)
{
    tokens = (T + kGroups - 1) / kGroups;
    groups = (T + tokens - 1) / tokens;
    parts = (groups + kChunks - 1) / kChunks;
}

bool sizes_ok(int64_t T, int64_t k, int64_t E)
{
    return T >= 0 && T <= INT32_MAX && k >= 1 && k <= MOE_SORT_MAX_K && E >= 1 && E <= kMaxE && T * k <= INT32_MAX;
}

// a launch that may begin while the one before it on the stream ends
cudaError_t launch_next(void (*kernel)(Params), unsigned grid, unsigned threads, int smem, cudaStream_t st, const Params &p)
{
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// threads of a token whose row is `columns` threads' work: a power of two up to 16, else warps, at most `most` and as few
// as take no more turns than those would
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

// The cluster and shared memory of sort_count and sort_index are beyond what a kernel may have unasked: asked for once on
// each device.
int index_smem(int64_t E) { return (int)((4 + 2 * (kCountThreads / 32)) * (E + 1)); }
int count_smem(int64_t E) { return (int)(4 * (kOfBlock + 1) * (E + 1)); }

cudaError_t allow_clusters()
{
    static std::atomic<uint64_t> done;
    mrr_device::Info info;
    if (!mrr_device::current(info))
        return cudaErrorUnknown;
    const uint64_t bit = info.device < mrr_device::kMaxDevices ? 1ull << info.device : 0;
    if (done.load(std::memory_order_acquire) & bit)
        return cudaSuccess;
    cudaError_t err = cudaSuccess;
    auto allow = [&](void (*kernel)(Params), int smem) {
        if (err == cudaSuccess)
            err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (err == cudaSuccess)
            err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    };
    allow(sort_count, count_smem(kMaxE));
    allow(sort_index, index_smem(kIndexE));
    if (err == cudaSuccess && bit)
        done.fetch_or(bit, std::memory_order_release);
    return err;
}

template <int W>
cudaError_t launch_few(const Params &p, cudaStream_t st)
{
    // where tokens are few, several blocks share a token's row, 1 KB each at least
    const int64_t most = (p.row_bytes + 1023) / 1024, want = kGroups / p.groups;
    const unsigned splits = (unsigned)(want < 1 || !p.out ? 1 : want < most ? want : most);
    sort_few<W><<<dim3(p.groups + 1, splits), kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_many(Params p, bool wide, cudaStream_t st)
{
    cudaError_t err = allow_clusters();
    if (err != cudaSuccess)
        return err;
    if (p.n <= kIndexSlots && p.E <= kIndexE) {
        Params q = p;
        q.parts = (int)((p.n + kCluster * kCountThreads - 1) / (kCluster * kCountThreads));
        sort_index<<<kCluster, kCountThreads, index_smem(p.E), st>>>(q);
        err = cudaGetLastError();
    } else {
        sort_count<<<kCluster, kCountThreads, count_smem(p.E), st>>>(p);
        err = cudaGetLastError();
        if (err == cudaSuccess)
            err = launch_next(sort_rank, (unsigned)p.groups, kThreads, 0, st, p);
    }
    if (err != cudaSuccess)
        return err;
    const int most = wide ? kMoveThreads : kAnyThreads;
    p.group = group_of(wide ? (p.row_bytes / 16 + kMoveAtOnce - 1) / kMoveAtOnce : (p.row_bytes + 31) / 16, most);
    p.move_tokens = most / p.group;
    const unsigned threads = p.group * p.move_tokens;   // whole warps
    const int64_t blocks = (p.T + p.move_tokens - 1) / p.move_tokens + kZeroBlocks;
    return wide ? launch_next(sort_move, (unsigned)blocks, threads, 0, st, p)
                : launch_next(sort_move_any, (unsigned)blocks, threads, p.move_tokens * any_space(p.row_bytes), st, p);
}

bool aligned(const void *p, uintptr_t n) { return (uintptr_t)p % n == 0; }

}  // namespace

extern "C" {

size_t moe_sort_workspace(int64_t T, int64_t k, int64_t E)
{
    if (!sizes_ok(T, k, E) || T * k <= kFewSlots)
        return 0;
    return (size_t)((4 * (kChunks * (E + 1) + 1) + 255) / 256 * 256);
}

mrr_status moe_sort_run(const void *expert_idx, int idx_is_i64, int64_t T, int64_t k, int64_t first_expert, int64_t E,
                        const void *x, int64_t row_bytes, int64_t row_stride, const void *scales,
                        int64_t scale_row_bytes, const void *weight, moe_dtype weight_dt, void *sorted_x,
                        void *sorted_scales, float *sorted_weight, int32_t *token_idx, int32_t *row_idx,
                        void *expert_num, int64_t expert_num_type, void *workspace, size_t workspace_bytes,
                        mrr_stream_t stream)
{
    if (weight && weight_dt != MOE_F16 && weight_dt != MOE_BF16 && weight_dt != MOE_F32)
        return MRR_ERR_DTYPE;
    if (expert_num_type != 0 && expert_num_type != 1)
        return MRR_ERR_ATTR;
    // (first_expert + E - 1 past int64: a key's subtraction would wrap)
    if (!sizes_ok(T, k, E) || first_expert > INT64_MAX - (E - 1) || row_bytes < 0 || row_bytes > (1 << 24) || row_stride < row_bytes ||
        (scales && (scale_row_bytes < 1 || scale_row_bytes > (1 << 20))))
        return MRR_ERR_SHAPE;
    if (!expert_num || (T > 0 && (!expert_idx || !token_idx || !row_idx || (row_bytes > 0 && (!x || !sorted_x)) ||
                                  (scales && !sorted_scales) || (weight && !sorted_weight))))
        return MRR_ERR_NULL;
    const uintptr_t idx_bytes = idx_is_i64 ? 8 : 4;
    if (!aligned(expert_idx, idx_bytes) || !aligned(expert_num, idx_bytes) || !aligned(token_idx, 4) ||
        !aligned(row_idx, 4) || (weight && (!aligned(weight, weight_dt == MOE_F32 ? 4 : 2) || !aligned(sorted_weight, 4))))
        return MRR_ERR_ALIGN;
    if (moe_sort_workspace(T, k, E) > 0 &&
        (!workspace || !aligned(workspace, 256) || workspace_bytes < moe_sort_workspace(T, k, E)))
        return MRR_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (cudaMemsetAsync(expert_num, 0, idx_bytes * (size_t)E, st) == cudaSuccess)
            return MRR_OK;
        (void)cudaGetLastError();
        return MRR_ERR_CUDA;
    }
    int64_t tokens, groups, parts;
    cut(T, tokens, groups, parts);
    Params p;
    memset(&p, 0, sizeof(p));
    p.idx = expert_idx;
    p.first = (uint64_t)first_expert;
    p.x = static_cast<const uint8_t *>(x);
    p.out = row_bytes > 0 ? static_cast<uint8_t *>(sorted_x) : nullptr;
    p.row_bytes = row_bytes;
    p.row_stride = row_stride;
    if (scales) {
        p.scales = static_cast<const uint8_t *>(scales);
        p.out_scales = static_cast<uint8_t *>(sorted_scales);
        p.scale_row_bytes = scale_row_bytes;
        p.scale_unit = scale_row_bytes % 4 == 0 && aligned(scales, 4) && aligned(sorted_scales, 4) ? 4 : 1;
    }
    if (weight) {
        p.weight = weight;
        p.weight_dt = weight_dt;
        p.out_weight = sorted_weight;
    }
    p.token_idx = token_idx;
    p.row_idx = row_idx;
    p.num = expert_num;
    p.table = static_cast<uint32_t *>(workspace);
    p.T = T;
    p.n = (uint32_t)(T * k);
    p.k = (int)k;
    p.E = (int)E;
    p.idx64 = idx_is_i64 != 0;
    p.cumsum = expert_num_type == 0;
    p.tokens = (int)tokens;
    p.groups = (int)groups;
    p.parts = (int)parts;
    // widest vectors that rows, stride and pointers are multiples of
    const uintptr_t all = p.out ? (uintptr_t)x | (uintptr_t)sorted_x | (uintptr_t)row_bytes | (T > 1 ? (uintptr_t)row_stride : 0)
                                : 0;
    cudaError_t err;
    if (T * k > kFewSlots)
        err = launch_many(p, all % 16 == 0, st);
    else
        err = all % 16 == 0  ? launch_few<16>(p, st)
              : all % 8 == 0 ? launch_few<8>(p, st)
              : all % 4 == 0 ? launch_few<4>(p, st)
              : all % 2 == 0 ? launch_few<2>(p, st)
                             : launch_few<1>(p, st);
    if (err == cudaSuccess)
        return MRR_OK;
    (void)cudaGetLastError();
    return MRR_ERR_CUDA;
}

}  // extern "C"
