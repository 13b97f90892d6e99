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
// so the copies need no barrier of the block.  Rows that do not fit twice (grad_h, which is read once, then stays out),
// that come in pieces of 2 bytes, or that have more than 20480 elements are loaded directly; the last have 8 chunks a thread, whose
// 64 sums are more than the 64 registers of 1024 threads hold beside the rest (2000 x 20484: 237 us, 2000 x 20480 92).  Accesses to shared memory are what the kernel has least to
// spare of (with the weight read from there too, 71 % of L1's throughput and 65 us for 8191 x 4100 bfloat16), so the
// weight is held in registers, and with one chunk a thread so are 16-bit rows, packed as they come.
// 8191 x 4100: 54.6 us; 16384 x 7168: 146 us, 6.4 TB/s; 4000 x 12288 float32: 137 us.
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
                auto fetch_one = [&](int t) {
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
                };
                // (a loop would keep `from` in local memory, and L1 has little room beside the stages)
                fetch_one(0);
                fetch_one(1);
                if (tensors == 3)
                    fetch_one(2);
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

// Threads of a block at most: of 2 chunks a thread 896 on an SM, whose registers give each 72 (16384 x 7172 by one block of
// 480 threads 167 us, by 256 threads of 4 chunks 308).
template <int NV, bool kBlock, int kPerSm>
constexpr int most_threads() { return !kBlock ? 32 * kShortWarps : NV == 1 ? 256 : NV == 2 ? 896 / kPerSm : NV == 4 ? 640 : 1024; }

// NV chunks a thread; kBlock: a block has a row at a time, else each of its warps has one.
template <int DT, int W, int NV, bool kBlock, int kPerSm, int kStages>
__global__ void __launch_bounds__(most_threads<NV, kBlock, kPerSm>(), kPerSm) rms_norm_grad(GradParams p)
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
    in.tensors = p.tensors;
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
                if (in.tensors == 3) {
                    in.get(stage, row, 2, i).get(d);
                } else {
                    Chunk<DT, W> c;
                    c.load(in.from[2] + row * in.size, (in.tid + i * in.threads) * Chunk<DT, W>::kBytes, in.size);
                    c.get(d);
                }
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

template <int DT, int W, int NV, bool kBlock, int kPerSm, int kStages>
cudaError_t launch(GradParams p, int tensors, unsigned threads, int smem, const mrr_device::Info &info, cudaStream_t st)
{
    static std::atomic<uint64_t> done;
    auto kernel = rms_norm_grad<DT, W, NV, kBlock, kPerSm, kStages>;
    const cudaError_t err = mrr_device::allow_smem(kernel, info, done);
    if (err != cudaSuccess)
        return err;
    p.tensors = tensors;
    kernel<<<(unsigned)grad_blocks(p.T, p.H), threads, kSumBytes + smem, st>>>(p);
    return cudaGetLastError();
}

template <int DT, int W, int NV, bool kBlock, int kPerSm>
cudaError_t launch(const GradParams &p, const mrr_device::Info &info, cudaStream_t st)
{
    const int chunks = (p.H + 7) / 8, all = p.grad_h ? 3 : 2;
    const unsigned threads = kBlock ? ((chunks + NV - 1) / NV + 31) / 32 * 32 : 32 * kShortWarps;
    const int row = NV * (int)threads * Chunk<DT, W>::kBytes;
    const int shares = kBlock ? 0 : kShortWarps * p.H * 4;   // in the stages' place, at the end
    auto bytes = [&](int stages, int tensors) {
        const int b = stages * tensors * row;
        return b > shares ? b : shares;
    };
    if constexpr (W > 2 && NV <= 4) {
        // two blocks on an SM, or one; pieces of less than 16 bytes come through L1 and leave it room (8191 x 4100: three
        // stages 55.9 us, two 54.9; 4000 x 12292: 122 and 100; 16384 x 1500: 41.5 and 45.5)
        const int whole = info.smem_max - 1024, most = W == 16 ? whole : 96 * 1024;
        if (bytes(3, all) <= (kPerSm == 2 ? most / 2 - 512 : most))
            return launch<DT, W, NV, kBlock, kPerSm, 3>(p, all, threads, bytes(3, all), info, st);
        if (bytes(2, all) <= whole)
            return launch<DT, W, NV, kBlock, kPerSm, 2>(p, all, threads, bytes(2, all), info, st);
        // without grad_h, which is read once
        if (bytes(2, 2) <= whole)
            return launch<DT, W, NV, kBlock, kPerSm, 2>(p, 2, threads, bytes(2, 2), info, st);
    }
    return launch<DT, W, NV, kBlock, kPerSm, 0>(p, all, threads, bytes(0, 0), info, st);
}

template <int DT, int W>
cudaError_t launch_grad(const GradParams &p, const mrr_device::Info &info, cudaStream_t st)
{
    const int chunks = (p.H + 7) / 8;
    return chunks <= 32     ? launch<DT, W, 1, false, 1>(p, info, st)
           : chunks <= 128  ? launch<DT, W, 4, false, 1>(p, info, st)
           : chunks <= 256  ? launch<DT, W, 1, true, 2>(p, info, st)
           : chunks <= 896  ? launch<DT, W, 2, true, 2>(p, info, st)
           : chunks <= 1792 ? launch<DT, W, 2, true, 1>(p, info, st)
           : chunks <= 2560 ? launch<DT, W, 4, true, 1>(p, info, st)
                            : launch<DT, W, 8, true, 1>(p, info, st);
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
