// The gradient of the root-mean-square norm (include/moe_norm.h).
//
// With g = grad_y weight, r = 1 / sqrt(mean(h^2) + eps):
//   grad_x = r g - h r^3 sum(g h) / H + grad_h,      grad_weight = sum over rows of grad_y h r
// Both sums over a row are of h and grad_y as they come from memory, so one joint sum over the row's threads gives
// r and the other factor, and a row is read once.  HBM bounds it.
//
// The blocks stay for many rows and hold their share of grad_weight in registers; each leaves one row of partial
// sums, which a second launch adds in order.  What a row waits for (its loads, the sum over the block) is hidden by
// copies that run kStages rows ahead into shared memory: each warp copies, and later reads, its own chunks only,
// so the copies need no barrier of the block.  Rows that do not fit, or that come in pieces of 2 bytes, are loaded
// directly.  Accesses to shared memory are what the kernel has least to spare of (with the weight read from there too,
// 71 % of L1's throughput and 65 us for 8191 x 4100 bfloat16), so the weight is held in registers, and with one chunk
// a thread so are 16-bit rows, packed as they come.  8191 x 4100: 53 us; 16384 x 7168: 142 us, 6.6 TB/s.
#pragma once

#include <atomic>

#include "column_sum.cuh"
#include "device_info.h"
#include "moe_norm.h"
#include "rms_norm.h"

namespace moe_norm {
namespace {

using namespace moe_rows;

constexpr int kSumWords = 32;     // most warps of a block
constexpr int kSumBytes = 2 * kSumWords * 8;

template <int W>
__device__ __forceinline__ void copy_async(void *to, const void *from)
{
    if (W == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mrr::smem_addr(to)), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(mrr::smem_addr(to)), "l"(from), "n"(W) : "memory");
}

// The chunks of h, grad_y and grad_h that a warp has of the rows ahead.  kStages 0: none, loaded when asked for.
template <int DT, int W, int NV, int kStages>
struct Ahead {
    using C = Chunk<DT, W>;
    const uint8_t *from[3];
    uint8_t *own;              // this thread's first slot
    int tid, threads, size, slots, tensors;

    __device__ __forceinline__ uint8_t *slot(int stage, int which, int i) const
    {
        return own + ((stage * tensors + which) * slots + i * threads) * C::kBytes;
    }

    // bytes past the row's end are zeros in every stage, and never copied
    __device__ __forceinline__ void clear() const
    {
        for (int s = 0; s < kStages; ++s)
            for (int t = 0; t < tensors; ++t)
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int b = 0; b < C::kBytes; b += 16)
                        *reinterpret_cast<uint4 *>(slot(s, t, i) + b) = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
    }

    // the warp's chunks, in pieces that follow each other from lane to lane
    __device__ __forceinline__ void fetch(int stage, int64_t row, int64_t T) const
    {
        if constexpr (kStages > 0) {
            __syncwarp();   // the stage's last row has been read
            if (row < T) {
                const int shift = tid % 32 * (W - C::kBytes);   // from this lane's chunk to its first piece
                for (int t = 0; t < tensors; ++t) {
                    const uint8_t *src = from[t] + row * size;
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int at = (tid + i * threads) * C::kBytes + shift;
                        uint8_t *to = slot(stage, t, i) + shift;
#pragma unroll
                        for (int b = 0; b < C::kBytes / W; ++b)
                            if (at + 32 * W * b < size)
                                copy_async<W>(to + 32 * W * b, src + at + 32 * W * b);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }

    __device__ __forceinline__ void wait() const
    {
        if constexpr (kStages > 0) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages > 0 ? kStages - 1 : 0) : "memory");
            __syncwarp();
        }
    }

    __device__ __forceinline__ C get(int stage, int64_t row, int which, int i) const
    {
        C c;
        if constexpr (kStages > 0) {
            const uint4 *q = reinterpret_cast<const uint4 *>(slot(stage, which, i));
#pragma unroll
            for (int b = 0; b < C::kBytes / 16; ++b) {
                const uint4 v = q[b];
                c.w[4 * b] = v.x, c.w[4 * b + 1] = v.y, c.w[4 * b + 2] = v.z, c.w[4 * b + 3] = v.w;
            }
        } else {
            c.load(from[which] + row * size, (tid + i * threads) * C::kBytes, size);
        }
        return c;
    }
};

// Threads of a block at most: of 2 chunks a thread 448, so that two blocks' registers (72 a thread) fit an SM.
template <int NV, bool kBlock>
constexpr int most_threads() { return !kBlock ? 32 * kShortWarps : NV == 2 ? 448 : NV <= 4 ? 512 : 1024; }

// NV chunks a thread; kBlock: a block has a row at a time, else each of its warps has one.
template <int DT, int W, int NV, bool kBlock, int kStages>
__global__ void __launch_bounds__(most_threads<NV, kBlock>(), NV > 2 || !kBlock ? 1 : 2) rms_norm_grad(GradParams p)
{
    // (all of it dynamic: together with static memory it could not be allowed up to the device's limit)
    extern __shared__ __align__(16) uint8_t memory[];
    float2 (*sums)[kSumWords] = reinterpret_cast<float2 (*)[kSumWords]>(memory);
    uint8_t *space = memory + kSumBytes;
    mrr::grid_launch_dependents();
    constexpr bool kHoldWeight = NV <= 4, kHoldRow = DT != MOE_F32 && NV == 1;
    const int warp = threadIdx.x / 32;
    const int64_t step = kBlock ? gridDim.x : gridDim.x * kShortWarps;
    Ahead<DT, W, NV, kStages> in;
    in.from[0] = static_cast<const uint8_t *>(p.h);
    in.from[1] = static_cast<const uint8_t *>(p.grad_y);
    in.from[2] = static_cast<const uint8_t *>(p.grad_h);
    in.tensors = p.grad_h ? 3 : 2;
    in.threads = kBlock ? blockDim.x : 32;
    in.tid = kBlock ? threadIdx.x : threadIdx.x % 32;
    in.size = p.H * Chunk<DT, W>::kElem;
    in.slots = NV * blockDim.x;
    in.own = space + (kBlock ? in.tid : NV * 32 * warp + in.tid) * Chunk<DT, W>::kBytes;
    in.clear();

    float acc[NV][8], weight[kHoldWeight ? NV : 1][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (kHoldWeight)
            load_weight<DT, W>(p.weight, p.weight_f32, in.tid + i * in.threads, p.H, weight[kHoldWeight ? i : 0]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            acc[i][j] = 0.0f;
    }
    const float per_element = 1.0f / (float)p.H;
    int64_t row = kBlock ? blockIdx.x : blockIdx.x * kShortWarps + warp;
    for (int s = 0; s < kStages; ++s)
        in.fetch(s, row + s * step, p.T);
    int turn = 0, stage = 0;
    for (; row < p.T; row += step, turn ^= 1) {
        in.wait();
        Chunk<DT, W> held[kHoldRow ? NV : 1][2];
        auto get = [&](int i, bool again, float (&h)[8], float (&g)[8]) {
            const int at = kHoldRow ? i : 0;
            if (!kHoldRow || !again) {
                held[at][0] = in.get(stage, row, 0, i);
                held[at][1] = in.get(stage, row, 1, i);
            }
            // (unpacked anew each time: kept as floats they would take twice the registers)
            if (kHoldRow && again) {
#pragma unroll
                for (int j = 0; j < Chunk<DT, W>::kWords; ++j)
                    asm volatile("" : "+r"(held[at][0].w[j]), "+r"(held[at][1].w[j]));
            }
            held[at][0].get(h);
            held[at][1].get(g);
            if (!kHoldWeight)
                load_weight<DT, W>(p.weight, p.weight_f32, in.tid + i * in.threads, p.H, weight[0]);
        };
        float squares = 0.0f, inner = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float h[8], g[8];
            get(i, false, h, g);
            const float (&w)[8] = weight[kHoldWeight ? i : 0];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                squares = fmaf(h[j], h[j], squares);
                inner = fmaf(g[j] * h[j], w[j], inner);
            }
        }
        squares = warp_sum(squares);
        inner = warp_sum(inner);
        if (kBlock) {
            // two sets of words in turn: one barrier a row
            if (threadIdx.x % 32 == 0)
                sums[turn][warp] = make_float2(squares, inner);
            __syncthreads();
            squares = inner = 0.0f;
            for (int w = 0; w < blockDim.x / 32; ++w) {
                squares += sums[turn][w].x;
                inner += sums[turn][w].y;
            }
        }
        const float r = rsqrtf(fmaf(squares, per_element, p.eps));
        const float factor = -(inner * per_element * r) * r * r;   // (r^3 alone passes float32 where eps is below 2^-85)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float h[8], g[8], d[8];
            get(i, true, h, g);
            const float (&w)[8] = weight[kHoldWeight ? i : 0];
            if (p.grad_h) {
                in.get(stage, row, 2, i).get(d);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    d[j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                acc[i][j] = fmaf(g[j] * h[j], r, acc[i][j]);
                d[j] = fmaf(g[j] * w[j], r, fmaf(h[j], factor, d[j]));
            }
            Chunk<DT, W> out;
            out.set(d);
            out.store(static_cast<uint8_t *>(p.grad_x) + row * in.size, (in.tid + i * in.threads) * Chunk<DT, W>::kBytes, in.size);
        }
        in.fetch(stage, row + kStages * step, p.T);
        stage = stage + 1 < kStages ? stage + 1 : 0;
    }
    if (!p.partial)
        return;
    float *to = p.partial + (int64_t)blockIdx.x * p.H;
    if (kBlock) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (8 * (in.tid + i * in.threads) + j < p.H)
                    to[8 * (in.tid + i * in.threads) + j] = acc[i][j];
    } else {
        // the warps' shares, in order; every copy has arrived by the wait of the last row
        float *shares = reinterpret_cast<float *>(space);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (8 * (in.tid + 32 * i) + j < p.H)
                    shares[warp * p.H + 8 * (in.tid + 32 * i) + j] = acc[i][j];
        __syncthreads();
        for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kShortWarps; ++w)
                s += shares[w * p.H + c];
            to[c] = s;
        }
    }
}

template <int DT, int W, int NV, bool kBlock, int kStages>
cudaError_t launch(const GradParams &p, unsigned threads, int smem, const mrr_device::Info &info, cudaStream_t st)
{
    static std::atomic<uint64_t> done;
    auto kernel = rms_norm_grad<DT, W, NV, kBlock, kStages>;
    const cudaError_t err = mrr_device::allow_smem(kernel, info, done);
    if (err != cudaSuccess)
        return err;
    kernel<<<(unsigned)grad_blocks(p.T, p.H), threads, kSumBytes + smem, st>>>(p);
    return cudaGetLastError();
}

template <int DT, int W, int NV, bool kBlock>
cudaError_t launch(const GradParams &p, const mrr_device::Info &info, cudaStream_t st)
{
    const int chunks = (p.H + 7) / 8;
    const unsigned threads = kBlock ? ((chunks + NV - 1) / NV + 31) / 32 * 32 : 32 * kShortWarps;
    const int stage = (p.grad_h ? 3 : 2) * NV * (int)threads * Chunk<DT, W>::kBytes;
    const int shares = kBlock ? 0 : kShortWarps * p.H * 4;   // in the stages' place, at the end
    auto bytes = [&](int stages) { return stages * stage > shares ? stages * stage : shares; };
    if constexpr (W > 2 && NV <= 4) {
        const int half = info.smem_max / 2 - 1024, whole = info.smem_max - 1024;   // two blocks on an SM, or one
        // (a fourth stage leaves L1 too little: 75 us where three take 58)
        if (bytes(3) <= half)
            return launch<DT, W, NV, kBlock, 3>(p, threads, bytes(3), info, st);
        if (bytes(2) <= whole)
            return launch<DT, W, NV, kBlock, 2>(p, threads, bytes(2), info, st);
    }
    return launch<DT, W, NV, kBlock, 0>(p, threads, bytes(0), info, st);
}

template <int DT, int W>
cudaError_t launch_grad(const GradParams &p, const mrr_device::Info &info, cudaStream_t st)
{
    const int chunks = (p.H + 7) / 8;
    return chunks <= 32     ? launch<DT, W, 1, false>(p, info, st)
           : chunks <= 128  ? launch<DT, W, 4, false>(p, info, st)
           : chunks <= 256  ? launch<DT, W, 1, true>(p, info, st)
           : chunks <= 896  ? launch<DT, W, 2, true>(p, info, st)
           : chunks <= 2048 ? launch<DT, W, 4, true>(p, info, st)
                            : launch<DT, W, 8, true>(p, info, st);
}

template <int DT>
cudaError_t launch_any(const GradParams &p, uintptr_t all, const mrr_device::Info &info, cudaStream_t st)
{
    return all % 16 == 0                     ? launch_grad<DT, 16>(p, info, st)
           : all % 8 == 0                    ? launch_grad<DT, 8>(p, info, st)
           : all % 4 == 0 || DT == MOE_F32   ? launch_grad<DT, 4>(p, info, st)
                                             : launch_grad<DT, DT == MOE_F32 ? 4 : 2>(p, info, st);
}

}  // namespace
}  // namespace moe_norm
