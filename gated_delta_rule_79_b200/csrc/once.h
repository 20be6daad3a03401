// Host-side: a kernel's shared-memory limit is raised once per device, not at every launch (a
// one-token call lasts about as long as the two driver calls this saves).
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace gdr {

// `done`: a static of the launching function, one bit a device.
template <typename K>
inline cudaError_t allow_smem(K kern, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace gdr
