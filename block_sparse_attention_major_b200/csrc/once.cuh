// Host side: checks that hold for as long as a device is there.
#pragma once

#include <atomic>
#include <cuda_runtime.h>
#include <stdint.h>

namespace bsa {

// Checks something once for each device (of the first 64; each time on others): what a device or a
// kernel is does not change, and asking again costs a launch's host time.
class OncePerDevice {
 public:
  template <typename F>
  cudaError_t operator()(F&& f) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (bit & done_.load(std::memory_order_acquire)) return cudaSuccess;
    e = f();
    if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

}  // namespace bsa
