// The norm and its gradient on float32 rows.
#include "rms_norm_grad_kernel.cuh"
#include "rms_norm_kernel.cuh"

namespace moe_norm {

cudaError_t norm_f32(const Params &p, uintptr_t all, cudaStream_t st) { return launch_any<MOE_F32>(p, all, st); }

cudaError_t norm_grad_f32(const GradParams &p, uintptr_t all, const mrr_device::Info &info, cudaStream_t st)
{
    return launch_any<MOE_F32>(p, all, info, st);
}

}  // namespace moe_norm
