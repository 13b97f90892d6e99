// The experts' product on expert-major MXFP4 rows (include/moe_mx.h).
//
// y[r, n] = sum_k x[r, k] w[e(r), n, k]; gated: silu(y_gate) * y_up; times row_weight.
#include "mx.cuh"
#include "ws_layout.h"

using namespace moe_mx;

namespace {

constexpr int kTile = 64, kStep = 32, kThreads = 256;

struct Params {
    const uint8_t *codes, *scales;
    int64_t A, K;
    const void *counts;
    int counts_i64, counts_prefix, E;
    const uint8_t *w_codes, *w_scales;
    int64_t N;
    const float *row_weight;
    void *out;
    int out_dt;
    uint8_t *out_scales;
    uint32_t *status;
};

__device__ __forceinline__ int64_t count_at(const Params &p, int e)
{
    return p.counts_i64 ? __ldg(static_cast<const long long *>(p.counts) + e)
                        : (int64_t)__ldg(static_cast<const int *>(p.counts) + e);
}

// one tile of 64 rows of one expert by 64 outputs, 4 x 4 of them a thread, from decoded 32-blocks
template <bool kGated>
__global__ void __launch_bounds__(kThreads) grouped_simple(Params p)
{
    constexpr int kMats = kGated ? 2 : 1;
    __shared__ float sx[kTile][kStep + 1], sw[kMats][kTile][kStep + 1], sy[kTile][kTile + 1];
    __shared__ int64_t s_row0, s_end;
    __shared__ int s_expert;
    if (threadIdx.x == 0) {
        int64_t at = 0, tile = blockIdx.x;
        int bad = 0;
        s_expert = -1;
        for (int e = 0; e < p.E; ++e) {
            const int64_t c = p.counts_prefix ? count_at(p, e) - at : count_at(p, e);
            if (c < 0 || c > p.A - at) {
                bad = c < 0 ? mrr_ws::kFlagNonPos : mrr_ws::kFlagSum;
                break;
            }
            const int64_t tiles = (c + kTile - 1) / kTile;
            if (s_expert < 0 && tile < tiles) {
                s_expert = e;
                s_row0 = at + tile * kTile;
                s_end = at + c;
            }
            tile -= tiles;
            at += c;
        }
        if (!bad && at != p.A)
            bad = mrr_ws::kFlagSum;
        if (bad)
            s_expert = -1;
        if (blockIdx.x == 0 && blockIdx.y == 0) {
            p.status[0] = bad;
            p.status[1] = 0;
        }
    }
    __syncthreads();
    if (s_expert < 0)
        return;
    const int64_t row0 = s_row0, end = s_end, n0 = (int64_t)blockIdx.y * kTile, srow = scale_row_bytes(p.K);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float acc[kMats][4][4] = {};
    for (int64_t k0 = 0; k0 < p.K; k0 += kStep) {
        for (int i = threadIdx.x; i < kTile * (1 + kMats) * 4; i += kThreads) {   // 8 elements each
            const int r = i / 4, part = i % 4, m = r / kTile - 1, rr = r % kTile;
            const uint8_t *q = p.codes, *s = p.scales;
            int64_t row = row0 + rr;
            bool in = row < end;
            if (m >= 0) {
                q = p.w_codes, s = p.w_scales;
                in = n0 + rr < p.N;
                row = ((int64_t)s_expert * kMats + m) * p.N + n0 + rr;
            }
            float v[8] = {};
            if (in) {
                decode8(__ldg(reinterpret_cast<const uint32_t *>(q + row * (p.K / 2) + k0 / 2) + part), v);
                const float f = e8m0_value(__ldg(s + row * srow + k0 / 32));
                for (int j = 0; j < 8; ++j)
                    v[j] *= f;
            }
            float *d = m < 0 ? &sx[rr][part * 8] : &sw[m < 0 ? 0 : m][rr][part * 8];
            for (int j = 0; j < 8; ++j)
                d[j] = v[j];
        }
        __syncthreads();
        for (int k = 0; k < kStep; ++k)
            for (int m = 0; m < kMats; ++m)
                for (int a = 0; a < 4; ++a)
                    for (int b = 0; b < 4; ++b)
                        acc[m][a][b] = fmaf(sx[ty + 16 * a][k], sw[m][tx + 16 * b][k], acc[m][a][b]);
        __syncthreads();
    }
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) {
            const int64_t row = row0 + ty + 16 * a, n = n0 + tx + 16 * b;
            float y = acc[0][a][b];
            if (kGated)
                y = y / (1.f + expf(-y)) * acc[kMats - 1][a][b];
            if (p.row_weight && row < end)
                y *= p.row_weight[row];
            sy[ty + 16 * a][tx + 16 * b] = y;
            if (row < end && n < p.N) {
                if (p.out_dt == MOE_F32)
                    store1<MOE_F32>(p.out, row * p.N + n, y);
                else if (p.out_dt == MOE_BF16)
                    store1<MOE_BF16>(p.out, row * p.N + n, y);
                else if (p.out_dt == MOE_F16)
                    store1<MOE_F16>(p.out, row * p.N + n, y);
            }
        }
    if (p.out_dt != MOE_MXFP4)
        return;
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * 2; i += kThreads) {   // one 32-block each; N is a multiple of 32
        const int r = i / 2, h = i % 2;
        const int64_t row = row0 + r, n = n0 + 32 * h;
        if (row >= end || n >= p.N)
            continue;
        uint32_t m = 0u;
        for (int j = 0; j < 32; ++j)
            m = max(m, __float_as_uint(sy[r][32 * h + j]) & 0x7fffffffu);
        const uint32_t sb = scale_byte(m);
        const float f = inverse_scale(sb);
        uint8_t *q = static_cast<uint8_t *>(p.out) + row * (p.N / 2) + n / 2;
        for (int j = 0; j < 16; ++j)
            q[j] = (uint8_t)encode2(sy[r][32 * h + 2 * j] * f, sy[r][32 * h + 2 * j + 1] * f);
        uint8_t *so = p.out_scales + row * scale_row_bytes(p.N) + n / 32;
        so[0] = (uint8_t)sb;
        if (n / 32 % 2 == 0 && n + 32 >= p.N)
            so[1] = 127;
    }
}

}  // namespace

extern "C" {

size_t moe_mx_grouped_workspace(int64_t E) { return E < 1 ? 0 : mrr_ws::kHeaderBytes; }

mrr_status moe_mx_grouped_run(const uint8_t *codes, const uint8_t *scales, int64_t A, int64_t K,
                              const void *expert_num, int expert_num_is_i64, int64_t expert_num_type, int64_t E,
                              const uint8_t *w_codes, const uint8_t *w_scales, int64_t N, int gated,
                              const float *row_weight, void *out, moe_dtype out_dt, uint8_t *out_scales,
                              void *workspace, size_t workspace_bytes, mrr_stream_t stream)
{
    if (out_dt != MOE_F16 && out_dt != MOE_BF16 && out_dt != MOE_F32 && out_dt != MOE_MXFP4)
        return MRR_ERR_DTYPE;
    if (expert_num_is_i64 != 0 && expert_num_is_i64 != 1)
        return MRR_ERR_DTYPE;
    if ((expert_num_type != 0 && expert_num_type != 1) || (gated != 0 && gated != 1))
        return MRR_ERR_ATTR;
    if (A < 0 || A > INT32_MAX || E < 1 || E > 4096 || K < 32 || K % 32 || K > (1 << 20) || N < 1 || N > (1 << 20) ||
        (out_dt == MOE_MXFP4 && N % 32))
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
    Params p{codes, scales, A, K, expert_num, expert_num_is_i64, expert_num_type == 0, (int)E, w_codes, w_scales, N,
             row_weight, out, (int)out_dt, out_scales, static_cast<uint32_t *>(workspace)};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t tiles = A / kTile + E;   // at least as many as the experts' tiles
    const dim3 grid((unsigned)tiles, (unsigned)((N + kTile - 1) / kTile));
    if (gated)
        grouped_simple<true><<<grid, kThreads, 0, s>>>(p);
    else
        grouped_simple<false><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? MRR_OK : MRR_ERR_CUDA;
}

}  // extern "C"
