// What a launch asks of the current device each time, asked of the driver once for each device: the
// calls behind it cost as much as a small kernel.
// What is remembered belongs to this copy of the library: functions that hold it in a static variable are
// static themselves, as the loader would make an inline function's variable one for all copies in a process,
// and a kernel's attributes are each copy's own.
#ifndef MRR_DEVICE_INFO_H
#define MRR_DEVICE_INFO_H

#include <atomic>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mrr_device {

constexpr int kMaxDevices = 64;

struct Info {
    int device, sms, smem_max;   // smem_max: most dynamic shared memory of a block (opt-in)
};

// the current device; false on a CUDA error
static inline bool current(Info &info)
{
    static std::atomic<int64_t> known[kMaxDevices];   // SMs << 32 | bytes, 0: not asked yet
    if (cudaGetDevice(&info.device) != cudaSuccess)
        return false;
    const bool keep = info.device >= 0 && info.device < kMaxDevices;
    int64_t v = keep ? known[info.device].load(std::memory_order_relaxed) : 0;
    if (v == 0) {
        if (cudaDeviceGetAttribute(&info.sms, cudaDevAttrMultiProcessorCount, info.device) != cudaSuccess ||
            cudaDeviceGetAttribute(&info.smem_max, cudaDevAttrMaxSharedMemoryPerBlockOptin, info.device) != cudaSuccess)
            return false;
        v = (int64_t)info.sms << 32 | info.smem_max;
        if (keep)
            known[info.device].store(v, std::memory_order_relaxed);
    }
    info.sms = (int)(v >> 32);
    info.smem_max = (int)(v & 0xffffffff);
    return true;
}

// allow `kernel` up to info.smem_max bytes of dynamic shared memory, once for each device; `done` is
// a static of the caller's, one for each kernel
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, const Info &info, std::atomic<uint64_t> &done)
{
    const uint64_t bit = info.device >= 0 && info.device < kMaxDevices ? 1ull << info.device : 0;
    if (done.load(std::memory_order_acquire) & bit)
        return cudaSuccess;
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, info.smem_max);
    if (err == cudaSuccess && bit)
        done.fetch_or(bit, std::memory_order_release);
    return err;
}

}  // namespace mrr_device

#endif  // MRR_DEVICE_INFO_H
