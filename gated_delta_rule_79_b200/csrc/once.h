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

// Launches `kern` so that its blocks may start before the kernel before it in the stream has
// finished; the kernel itself waits (griddepcontrol.wait) before it reads what that one wrote.
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kern)(P...), dim3 grid, int threads, int smem,
                                cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace gdr
