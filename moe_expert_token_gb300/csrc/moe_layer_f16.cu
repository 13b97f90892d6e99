// Instances of the layer's kernel for x in f16 (each type's and form's compile beside the others').
#include "moe_layer_kernel.cuh"

namespace moe_layer {

cudaError_t launch_f16(const Params &p, bool mx, int regime, const mrr_device::Info &info, int grid, size_t smem,
                       cudaStream_t s)
{
    return launch_dt<MOE_F16, false>(p, mx, regime, info, grid, smem, s);
}

}  // namespace moe_layer
