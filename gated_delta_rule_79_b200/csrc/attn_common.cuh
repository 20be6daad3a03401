// Softmax attention with a sliding window and sinks: what its kernels share.
//
// "Super Apriel: One Checkpoint, Many Speeds", §2A (Mixer Vocabulary) names full and
// sliding-window attention beside the recurrent mixers.  Query i of Tq sits at position
// p = Tk - Tq + i and sees key j when j <= p, j and p lie before the sequence's length, and
// p - j < window (0: no window) or j < sinks:
//
//     s_ij = scale q_i.k_j,   lse_i = log sum_j e^(s_ij),   o_i = sum_j e^(s_ij - lse_i) v_j
//
// A query that sees nothing has o = 0 and lse = -inf.  Gradients, with D_i = do_i . o_i:
//
//     p_ij = e^(s_ij - lse_i),   ds_ij = scale p_ij (do_i . v_j - D_i)
//     dv_j = sum_i p_ij do_i,    dq_i = sum_j ds_ij k_j,    dk_j = sum_i ds_ij q_i
#pragma once

#include "common.cuh"
#include "launch.h"

namespace gdr {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
// The mask of one sequence.  window > 0, or 0 for none; sinks is 0 without a window.
struct Mask {
  int off;      // position of query 0
  int len;      // keys and queries at and past this position do not count
  int window, sinks;
};

__device__ __forceinline__ Mask make_mask(const int* lengths, int b, int Tq, int Tk, int window,
                                          int sinks) {
  Mask m;
  m.off = Tk - Tq;
  m.len = lengths ? min(max(lengths[b], 0), Tk) : Tk;
  m.window = window;
  m.sinks = sinks;
  return m;
}

// Bits 0 .. h.
__device__ __forceinline__ uint32_t columns_to(int h) {
  return h < 0 ? 0u : 0xffffffffu >> (31 - min(h, 31));
}
// A query's visible keys as column thresholds of a tile that starts at key j0: column c is
// visible when c <= hi and (c >= lo or c < sink).  hi < 0 hides everything.
struct RowCols {
  int hi, lo, sink;
  __device__ __forceinline__ bool sees(int c) const {
    return (c <= hi) & ((c >= lo) | (c < sink));
  }
  // columns c0 .. c0 + 31 as bits
  __device__ __forceinline__ uint32_t bits(int c0) const {
    return columns_to(hi - c0) & (~columns_to(lo - 1 - c0) | columns_to(sink - 1 - c0));
  }
};
// The elements of x, a row's columns, that are not visible become `hidden`: a test of one bit and
// a select each.  (Three comparisons an element made masked tiles two to four times as long.)
template <int N>
__device__ __forceinline__ void hide(float (&x)[N], const RowCols& rc, float hidden) {
#pragma unroll
  for (int q = 0; q < N / 32; ++q) {
    const uint32_t see = rc.bits(32 * q);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!(see & (1u << e))) x[32 * q + e] = hidden;
  }
}
__device__ __forceinline__ RowCols row_cols(const Mask& m, int p, int j0) {
  RowCols r;
  r.hi = p < m.len ? p - j0 : -1;      // p < len covers j < len as well
  r.lo = m.window ? p - m.window + 1 - j0 : -0x40000000;
  r.sink = m.sinks - j0;
  return r;
}
// The other way round: the queries that see key j, as thresholds of columns that start at
// position p0.
__device__ __forceinline__ RowCols col_rows(const Mask& m, int j, int p0) {
  RowCols r;
  r.lo = j - p0;
  r.hi = m.len - 1 - p0;
  if (m.window && j >= m.sinks) r.hi = min(r.hi, j - p0 + m.window - 1);
  r.sink = 0;
  return r;
}
// Whether the queries p0 .. p1 all see all of the keys j0 .. j1.
__device__ __forceinline__ bool all_visible(const Mask& m, int p0, int p1, int j0, int j1) {
  return j1 <= p0 && p1 < m.len && (m.window == 0 || p1 - j0 < m.window || j1 < m.sinks);
}

// Key tiles of BN keys that the queries i0 .. i1 see: tiles 0 .. nsink-1 hold sinks that lie
// before the window's first tile lo; then lo .. lo + nwin - 1.
struct KeyTiles {
  int nsink, lo, nwin;
  __device__ __forceinline__ int count() const { return nsink + nwin; }
  __device__ __forceinline__ int tile(int x) const { return x < nsink ? x : lo + x - nsink; }
  __device__ __forceinline__ bool has(int tl) const {
    return tl < nsink || (tl >= lo && tl < lo + nwin);
  }
};
template <int BN>
__device__ __forceinline__ KeyTiles key_tiles(const Mask& m, int i0, int i1) {
  KeyTiles t{0, 0, 0};
  const int p0 = max(m.off + i0, 0), p1 = min(m.off + i1, m.len - 1);
  if (p1 < p0) return t;
  const int first = m.window ? max(0, p0 - m.window + 1) : 0;
  t.lo = first / BN;
  t.nwin = p1 / BN - t.lo + 1;
  t.nsink = min((m.sinks + BN - 1) / BN, t.lo);
  return t;
}

// Queries that see any of the keys j0 .. j1: i in [lo, hi) (empty when hi <= lo).
__device__ __forceinline__ void query_range(const Mask& m, int j0, int j1, int Tq, int& lo,
                                            int& hi) {
  lo = max(0, j0 - m.off);
  long last = (long)m.len - 1;
  if (m.window && j0 >= m.sinks) last = min(last, (long)j1 + m.window - 1);
  hi = j0 < m.len ? (int)min((long)Tq, last - m.off + 1) : 0;
}

}  // namespace attn
}  // namespace gdr
