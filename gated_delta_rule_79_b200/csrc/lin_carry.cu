// Linear attention: from what every segment leaves in the state to the state every segment is
// entered with (lin_common.cuh).  A thread carries four elements of a state through the
// segments, in place:
//
//     entering 0 = S_in,   entering 1 = a^(n_0 - 1 + e0) S_in + left 0,
//     entering p+1 = a^(n_p) entering p + left p
//
// (S_in is copied as well: the last segment may write the final state over it while the first
// one has yet to start.)
// Bound by memory latency and, at 8 bytes an element and segment, by L2; the reads do not wait
// for one another.

#include "lin_common.cuh"
#include "once.h"

namespace gdr {
namespace {

using namespace lin;

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
lin_carry_kernel(const LinScan sc) {
  const LinJob& jb = sc.job[blockIdx.y];
  const int size = sc.dk * sc.dv, blocks = size / (4 * kThreads);
  const int bh = blockIdx.x / blocks, h = bh % sc.H;
  const int e = (blockIdx.x % blocks * kThreads + threadIdx.x) * 4;
  const double l2 = log2_decay(sc.decay[h]);
  let_next_start();
  // elements e .. e + 3 are (r, c) .. (r, c + 3)
  float S[4] = {0.f, 0.f, 0.f, 0.f};
  if (jb.s_in) {
    const float* s = jb.s_in + (size_t)bh * size;
    const int r = sc.part_rows ? e / sc.dk : e / 4 % sc.dv;
    const int c = sc.part_rows ? e % sc.dk : e / 4 / sc.dv * 4;
    if (jb.s_trans) {
#pragma unroll
      for (int i = 0; i < 4; ++i) S[i] = s[(size_t)(c + i) * sc.dv + r];
    } else {
      const float4 x = *reinterpret_cast<const float4*>(s + (size_t)r * sc.dk + c);
      S[0] = x.x, S[1] = x.y, S[2] = x.z, S[3] = x.w;
    }
  }
  float* part = sc.part + ((size_t)blockIdx.y * sc.B * sc.H + bh) * sc.nseg * size + e;
  // all segments but the one at the tensor's end are seg_len long; a decay as a pair of floats,
  // since its rounding would be the same in every segment and add up
  const Segment s0 = segment(0, jb.rev, sc.T, sc.seg_len, sc.nseg);
  const double d0 = decay_pow(l2, (long)s0.n - 1 + jb.e0), d1 = decay_pow(l2, sc.seg_len);
  const float h0 = (float)d0, l0 = (float)(d0 - (double)h0);
  const float h1 = (float)d1, l1 = (float)(d1 - (double)h1);
  wait_for_previous();
  *reinterpret_cast<float4*>(part) = make_float4(S[0], S[1], S[2], S[3]);
  part += size;
  constexpr int AHEAD = 8;          // reads in flight
  for (int p0 = 0; p0 < sc.nseg - 1; p0 += AHEAD) {
    float4 x[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (p0 + i < sc.nseg - 1) x[i] = *reinterpret_cast<const float4*>(part + (size_t)(p0 + i) * size);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (p0 + i < sc.nseg - 1) {
        const float fh = p0 + i ? h1 : h0, fl = p0 + i ? l1 : l0;
        S[0] = fmaf(fh, S[0], fmaf(fl, S[0], x[i].x));
        S[1] = fmaf(fh, S[1], fmaf(fl, S[1], x[i].y));
        S[2] = fmaf(fh, S[2], fmaf(fl, S[2], x[i].z));
        S[3] = fmaf(fh, S[3], fmaf(fl, S[3], x[i].w));
        *reinterpret_cast<float4*>(part + (size_t)(p0 + i) * size) =
            make_float4(S[0], S[1], S[2], S[3]);
      }
  }
}

}  // namespace

cudaError_t launch_lin_carry(const LinScan& sc, cudaStream_t st) {
  const int blocks = sc.dk * sc.dv / (4 * kThreads);
  return launch_after(lin_carry_kernel, dim3((unsigned)(sc.B * sc.H * blocks), sc.njobs), kThreads,
                      0, st, sc);
}

}  // namespace gdr
