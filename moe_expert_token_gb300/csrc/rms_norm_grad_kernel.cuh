// The gradient of the root-mean-square norm (include/moe_norm.h).
//
// With g = grad_y weight, r = 1 / sqrt(mean(h^2) + eps):
//   grad_x = r g - h r^3 sum(g h) / H + grad_h,      grad_weight = sum over rows of grad_y h r
// Both sums over a row are of h and grad_y as they come from memory, so one joint sum over the row's threads gives
// r and the other factor, and a row is read once.  HBM bounds it.
//
// The blocks stay for many rows and hold their share of grad_weight in registers; each leaves one row of partial
// sums, which a second launch adds in order.  What a row waits for (its loads, the sum over the block) is hidden by
// copies that run kStages rows ahead into shared memory: each thread copies, and later reads, its own chunks only,
// so the copies need no barrier.  Rows that do not fit, or that come in pieces of 2 bytes, are loaded directly.
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

// The chunks of h, grad_y and grad_h that a thread has of the rows ahead.  kStages 0: none, loaded when asked for.
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
    }

    __device__ __forceinline__ void fetch(int stage, int64_t row, int64_t T) const
    {
        if constexpr (kStages > 0) {
            if (row < T) {
                for (int t = 0; t < tensors; ++t) {
                    const uint8_t *src = from[t] + row * size;
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int at = (tid + i * threads) * C::kBytes;
#pragma unroll
                        for (int b = 0; b < C::kBytes; b += W)
                            if (at + b < size)
                                copy_async<W>(slot(stage, t, i) + b, src + at + b);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }

    __device__ __forceinline__ void wait() const
    {
        if constexpr (kStages > 0)
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages > 0 ? kStages - 1 : 0) : "memory");
    }

    __device__ __forceinline__ void get(int stage, int64_t row, int which, int i, float (&v)[8]) const
    {
        C c;
        if constexpr (kStages > 0) {
            const uint4 *q = reinterpret_cast<const uint4 *>(slot(stage, which, i));
#pragma unroll
            for (int b = 0; b < C::kBytes / 16; ++b)
                c.w[4 * b] = q[b].x, c.w[4 * b + 1] = q[b].y, c.w[4 * b + 2] = q[b].z, c.w[4 * b + 3] = q[b].w;
        } else {
            c.load(from[which] + row * size, (tid + i * threads) * C::kBytes, size);
        }
        c.get(v);
    }
};

// NV chunks a thread; kBlock: a block has a row at a time, else each of its warps has one.
template <int DT, int W, int NV, bool kBlock, int kStages>
__global__ void __launch_bounds__(kBlock ? (NV > 4 ? 1024 : 512) : 32 * kShortWarps, NV > 4 || !kBlock ? 1 : 2) rms_norm_grad(GradParams p)
{
    // (all of it dynamic: together with static memory it could not be allowed up to the device's limit)
    extern __shared__ __align__(16) uint8_t memory[];
    float2 (*sums)[kSumWords] = reinterpret_cast<float2 (*)[kSumWords]>(memory);
    uint8_t *space = memory + kSumBytes;
    mrr::grid_launch_dependents();
    constexpr bool kWeightHere = NV <= 4;   // up to 64 KB
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
    in.own = space + (kWeightHere ? 32 * in.slots : 0) + (kBlock ? in.tid : NV * 32 * warp + in.tid) * Chunk<DT, W>::kBytes;
    in.clear();

    // the weight of this thread's chunks as floats, in two planes of 16 bytes a chunk
    float4 *weight = reinterpret_cast<float4 *>(space) + (kBlock ? in.tid : NV * 32 * warp + in.tid);
    float acc[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (kWeightHere) {
            float w[8];
            load_weight<DT, W>(p.weight, p.weight_f32, in.tid + i * in.threads, p.H, w);
            weight[i * in.threads] = make_float4(w[0], w[1], w[2], w[3]);
            weight[in.slots + i * in.threads] = make_float4(w[4], w[5], w[6], w[7]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            acc[i][j] = 0.0f;
    }
    // h, grad_y and the weight of chunk i; read twice a row, which costs less than the threads that registers would
    auto get = [&](int stage, int64_t row, int i, float (&h)[8], float (&g)[8], float (&w)[8]) {
        in.get(stage, row, 0, i, h);
        in.get(stage, row, 1, i, g);
        if (kWeightHere) {
            const float4 lo = weight[i * in.threads], hi = weight[in.slots + i * in.threads];
            w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w, w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
        } else {
            load_weight<DT, W>(p.weight, p.weight_f32, in.tid + i * in.threads, p.H, w);
        }
    };
    const float per_element = 1.0f / (float)p.H;
    int64_t row = kBlock ? blockIdx.x : blockIdx.x * kShortWarps + warp;
    for (int s = 0; s < kStages; ++s)
        in.fetch(s, row + s * step, p.T);
    int turn = 0, stage = 0;
    for (; row < p.T; row += step, turn ^= 1) {
        in.wait();
        float squares = 0.0f, inner = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float h[8], g[8], w[8];
            get(stage, row, i, h, g, w);
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
        const float factor = -r * r * r * (inner * per_element);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float h[8], g[8], w[8], d[8];
            get(stage, row, i, h, g, w);
            if (p.grad_h) {
                in.get(stage, row, 2, i, d);
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
    const int slots = NV * (int)threads, stage = (p.grad_h ? 3 : 2) * slots * Chunk<DT, W>::kBytes;
    const int weight = NV <= 4 ? 32 * slots : 0;
    const int shares = kBlock ? 0 : kShortWarps * p.H * 4;   // in the place of the rest, at the end
    auto bytes = [&](int stages) { return weight + stages * stage > shares ? weight + stages * stage : shares; };
    if constexpr (W > 2 && NV <= 4) {
        const int half = info.smem_max / 2 - 1024, whole = info.smem_max - 1024;   // two blocks on an SM, or one
        if (bytes(4) <= half)
            return launch<DT, W, NV, kBlock, 4>(p, threads, bytes(4), info, st);
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
           : chunks <= 512  ? launch<DT, W, 1, true>(p, info, st)
           : chunks <= 1024 ? launch<DT, W, 2, true>(p, info, st)
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
