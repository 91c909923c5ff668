// Host helpers of kernel launches.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

namespace qg {

// Sets a kernel's attribute once per device (`done`: a bit for each of the
// first 64, set after the call succeeded; a concurrent first call sets it twice,
// which is harmless).
template <class Kernel>
cudaError_t set_once(std::atomic<uint64_t>& done, Kernel kernel, cudaFuncAttribute attribute, int value) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, attribute, value);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}
template <class Kernel>
cudaError_t set_smem_once(std::atomic<uint64_t>& done, Kernel kernel, int bytes) {
    return set_once(done, kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace qg
