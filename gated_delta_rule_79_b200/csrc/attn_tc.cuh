// What the tensor-core attention kernels share: operand descriptors of the bf16 tiles, the
// row thresholds of the mask, packed fp32 arithmetic, bounded waits.
//
// A tile is 128 (or 64) tokens of one head as TMA leaves it: D / 64 panels of `rows` rows x
// 128 bytes, 128-byte swizzled.  The same bytes serve as a K-major operand (the reduction
// runs over the channels: q k^T, do v^T) and as an MN-major one (it runs over the tokens:
// p v, ds k, ds^T q, p^T do), so nothing is transposed or copied.
#pragma once

#include <stdlib.h>

#include "attn_common.cuh"
#include "tc.cuh"

namespace gdr {
namespace attn {

using namespace tc;

constexpr uint32_t kDrain = 1u << 26;       // polls while draining work in flight

inline uint32_t attn_spin_limit() {
  const char* e = getenv("GDR_SPIN_LIMIT");
  if (!e || !*e) return 1u << 24;
  return (uint32_t)strtoul(e, nullptr, 10);
}

// K-major operand: 16 channels of k-step ks.  Panels of `rows` rows; 8-row groups 1024 bytes
// apart.
__device__ __forceinline__ uint64_t kmajor(uint32_t tile, int rows, int ks) {
  return sdesc(tile + (uint32_t)(ks >> 2) * rows * 128 + (ks & 3) * 32, 16, 1024);
}
// MN-major operand: 16 tokens of k-step ks, all D channels as the M or N index.  The panels
// of 64 channels lie rows * 128 bytes apart, 8-token groups 1024 bytes.
__device__ __forceinline__ uint64_t mnmajor(uint32_t tile, int rows, int ks) {
  return sdesc(tile + (uint32_t)ks * 2048, (uint32_t)rows * 128, 1024);
}
__host__ __device__ constexpr uint32_t idesc_bf16_mn(int M, int N) {   // B is MN-major
  return idesc_bf16(M, N) | (1u << 16);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float pack2(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<float*>(&p);
}

// Bounded waits of one CTA, made by whole warps: every lane gets the same answer.  The first
// warp to give up records it and raises the flag that ends the others.
struct Waits {
  unsigned int* status;
  volatile int* abort;
  uint32_t limit;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    for (uint32_t i = 0; i < limit; ++i) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
      if ((i & 63u) == 63u && __any_sync(0xffffffffu, *abort != 0)) return false;
    }
    atomicOr(status, 1u);
    *abort = 1;
    return false;
  }
};

template <int N> __device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N));
}
template <int N> __device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N));
}

// Rows r0 .. rows-1 of a tile set to zero by one warp, for operands whose reduction runs over
// the tokens: what lies behind a sequence's length may be NaN and would meet a weight of 0.
template <int D>
__device__ __forceinline__ void zero_rows(unsigned char* tile, int rows, int r0, int lane) {
  const uint4 z = make_uint4(0, 0, 0, 0);
  for (int pn = 0; pn < D / 64; ++pn)
    for (int e = r0 * 8 + lane; e < rows * 8; e += 32)
      *reinterpret_cast<uint4*>(tile + pn * rows * 128 + e * 16) = z;
  fence_smem_to_async();
  __syncwarp();
}

}  // namespace attn
}  // namespace gdr
