// The dynamic shared memory a kernel may use is set once per device: the call
// costs about a microsecond, as much as a tenth of a decode step's launch.
#pragma once

#include <atomic>
#include <cuda_runtime.h>

namespace csa {

class SmemOnce {
 public:
  template <typename F>
  cudaError_t operator()(F* kernel, size_t bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (bit != 0 && (done_.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<unsigned long long> done_{0};   // bit: device
};

}  // namespace csa
