// The norm and its gradient on float16 rows.
#include "rms_norm_grad_kernel.cuh"
#include "rms_norm_kernel.cuh"

namespace moe_norm {

cudaError_t norm_f16(const Params &p, uintptr_t all, cudaStream_t st) { return launch_any<MOE_F16>(p, all, st); }

cudaError_t norm_grad_f16(const GradParams &p, uintptr_t all, const mrr_device::Info &info, cudaStream_t st)
{
    return launch_any<MOE_F16>(p, all, info, st);
}

}  // namespace moe_norm
