// Linear attention with one decay per head: what its kernels share.
//
// A token mixer with a state of fixed size, like the two that "Super Apriel: One Checkpoint, Many
// Speeds", §2A (Mixer Vocabulary) names (GDN and KDA), but without the delta rule's correction;
// the paper does not name this one.  For every (sequence, head), with the decay a of that head,
//
//     S_t = a S_{t-1} + v_t k_t^T,      o_t = S_t q_t                       (S: d_v x d_k)
//
// Chunk-wise (tokens i = 0 .. L-1 of a chunk entered with state S):
//
//     o_i = a^(i+E) S q_i + sum_{j<=i} a^(i-j) (q_i . k_j) v_j
//     S'  = a^(L-1+E) S + sum_j a^(L-1-j) v_j k_j^T
//
// with E = 1.  The gradients are three scans of this same form over other tensors.  With
// G_t = a G_{t+1} + do_t q_t^T (the last one entered with dL/dS_T),
//
//     dq_t = S_t^T do_t      the scan of (q, k, v) := (do, v, k), entered with S_0^T
//     dv_t = G_t k_t         the scan of (k, q, do) from the last token to the first,
//                            entered with dL/dS_T; dL/dS_0 = a G_1 is a times its end state
//     dk_t = G_t^T v_t       the scan of (v, do, q), likewise, entered with (dL/dS_T)^T
//
// In the two reversed scans the entering state meets the first processed token undecayed:
// E = 0 in their first chunk (e0 below), 1 after it.
//
// A call is cut along the tokens into nseg segments of seg_len tokens, so that few (batch,
// head) pairs still fill the GPU: a first kernel forms what each segment but the last leaves in
// the state, a second one (lin_carry.cu) runs through the segments and turns that into the
// state each of them is entered with, a third one writes the outputs.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace gdr {
namespace lin {

// log2 of the decay in fp64; 0 and below act as an exact 0 for every power but the 0th
__device__ __forceinline__ double log2_decay(float a) {
  return a > 0.f ? log2((double)a) : -4096.0;
}
// a^n for n >= 0.  The exponent is formed in fp64: a product of fp32 powers would drift
// over the thousands of chunks that a decay near 1 reaches across.
__device__ __forceinline__ double decay_pow(double l2, long n) { return exp2(l2 * (double)n); }

// One segment in processing order: its first token and its length.
struct Segment {
  int a, n;
};
__device__ __forceinline__ Segment segment(int p, int rev, int T, int seg_len, int nseg) {
  const int r = rev ? nseg - 1 - p : p;
  Segment s;
  s.a = r * seg_len;
  s.n = min(seg_len, T - s.a);
  return s;
}

// Where element (r, c) of a d_v x d_k state lies in the workspace: four neighbours of a row
// together and rows next to each other, because the tensor-core kernels hold a row a thread.
__host__ __device__ __forceinline__ int part_at(int dv, int r, int c) {
  return ((c >> 2) * dv + r) * 4 + (c & 3);
}

}  // namespace lin
}  // namespace gdr
