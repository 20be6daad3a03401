// Key tiles whose gradients several CTAs sum (attn_tc_backward.cu, attn_simt.cu).
//
// dk and dv of a tile of A keys of a key head sum over all queries that see it, of every query
// head of the group: `steps` tiles of S queries.  Where that is far more than an SM's share (few
// key tiles, early ones without a window, one with sinks) the steps are cut into parts, a CTA
// each, whose fp32 sums a small kernel adds in order, so results do not depend on scheduling.
#pragma once

#include "attn_common.cuh"

namespace gdr {
namespace attn {

// Tiles [0, nfirst), those with sinks, are cut into up to pfirst parts of up to `cfirst` steps, the
// others into up to prest of up to `crest`.
struct Parts {
  int nfirst, pfirst, prest, cfirst, crest, ntiles;
  __host__ __device__ int items() const { return nfirst * pfirst + (ntiles - nfirst) * prest; }
  __device__ void locate(int item, int& tile, int& part) const {
    if (item < nfirst * pfirst) {
      tile = item / pfirst, part = item % pfirst;
    } else {
      const int r = item - nfirst * pfirst;
      tile = nfirst + r / prest, part = r % prest;
    }
  }
  __device__ int used(int steps, int tile) const {
    const int cap = tile < nfirst ? cfirst : crest, most = tile < nfirst ? pfirst : prest;
    return max(1, min(most, (steps + cap - 1) / cap));
  }
  bool cut() const { return pfirst > 1 || prest > 1; }
};

// The steps of a key tile: tiles of S queries from the lo-th, nt of them for each head.
template <int A, int S>
__device__ __forceinline__ void tile_steps(const Mask& m, int j0, int Tk, int Tq, int& lo,
                                           int& nt) {
  int first, hi;
  query_range(m, j0, min(j0 + A, Tk) - 1, Tq, first, hi);
  lo = first / S;
  nt = hi > first ? (hi + S - 1) / S - lo : 0;
}

// Where channel c of a part's dv (w = 0) or dk row lies: 8 channels of all rows next to each
// other, so that a thread a row and a thread a piece both touch whole lines.
__host__ __device__ __forceinline__ size_t part_at(const AttnArgs& f, int A, int D, int item, int bh,
                                                   int w, int row, int c) {
  return ((((size_t)item * f.B * f.Hkv + bh) * 2 + w) * (D / 8) + (c >> 3)) * A * 8 + row * 8 +
         (c & 7);
}

// The parts' sums added in order: 8 channels of a row a thread.
template <typename T, int D, int A, int S>
__global__ void __launch_bounds__(256)
attn_dkv_join(const AttnGradArgs a, const Parts parts) {
  const AttnArgs& f = a.f;
  constexpr int BLOCKS = A * (D / 8) * 2 / 256;
  const int at = blockIdx.x / BLOCKS;
  const int bh = at % (f.B * f.Hkv), tile = at / (f.B * f.Hkv);
  const int b = bh / f.Hkv, hk = bh % f.Hkv;
  const int j0 = tile * A;
  const Mask m = make_mask(f.lengths, b, f.Tq, f.Tk, f.window, f.sinks);
  int lo, nt;
  tile_steps<A, S>(m, j0, f.Tk, f.Tq, lo, nt);
  const bool head = tile < parts.nfirst;
  const int used = parts.used(f.Hq / f.Hkv * nt, tile);
  if (used == 1) return;
  const int item = head ? tile * parts.pfirst
                        : parts.nfirst * parts.pfirst + (tile - parts.nfirst) * parts.prest;
  const size_t step = (size_t)f.B * f.Hkv * 2 * A * D;       // from a part to the next
  const int e = blockIdx.x % BLOCKS * 256 + threadIdx.x;
  const int w = e / (A * (D / 8)), row = e % A, c = e / A % (D / 8) * 8;
  if (j0 + row >= f.Tk) return;
  const float* src = a.part + part_at(f, A, D, item, bh, w, row, c);
  alignas(16) T y[8];
  float x[8] = {};
#pragma unroll 4
  for (int p = 0; p < used; ++p) {
    const float4 u = *reinterpret_cast<const float4*>(src + p * step);
    const float4 v = *reinterpret_cast<const float4*>(src + p * step + 4);
    x[0] += u.x, x[1] += u.y, x[2] += u.z, x[3] += u.w;
    x[4] += v.x, x[5] += v.y, x[6] += v.z, x[7] += v.w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) Elem<T>::store(y + i, x[i]);
  T* dst = (T*)(w ? a.dk : a.dv) + (((size_t)b * f.Tk + j0 + row) * f.Hkv + hk) * D + c;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(y)[i];
}

template <typename T, int D, int A, int S>
cudaError_t launch_dkv_join(const AttnGradArgs& a, const Parts& p, cudaStream_t st) {
  if (!p.cut()) return cudaSuccess;
  const unsigned tiles = (unsigned)(p.prest > 1 ? p.ntiles : p.nfirst);
  attn_dkv_join<T, D, A, S>
      <<<tiles * (unsigned)(a.f.B * a.f.Hkv) * (A * (D / 8) * 2 / 256), 256, 0, st>>>(a, p);
  return cudaGetLastError();
}

// Steps of a key tile when every sequence is whole (the host's tile_steps).
template <int A, int S>
long host_steps(const AttnArgs& f, int tile) {
  const long off = (long)f.Tk - f.Tq, j0 = (long)tile * A;
  const long j1 = (j0 + A < f.Tk ? j0 + A : f.Tk) - 1;
  const long lo = j0 - off > 0 ? j0 - off : 0;
  long last = f.Tk - 1;
  if (f.window && j0 >= f.sinks && j1 + f.window - 1 < last) last = j1 + f.window - 1;
  const long hi = f.Tq < last - off + 1 ? f.Tq : last - off + 1;
  return hi > lo ? ((hi + S - 1) / S - lo / S) * (f.Hq / f.Hkv) : 0;
}

// For a GPU with places for `ctas` of the kernel's CTAs.  The cap is one and a half times the mean
// number of steps of a place: dq runs beside or after the last ones, and parts cost a pass of
// fp32 sums through memory.  Measured with 128-key tiles (32 heads, 8 key heads, d = 128): 256
// tokens 22 us against 31 uncut, 1024 tokens 69 and 107; factors of 1.25 and 2.5 were up to 25 %
// slower with windows of 512 and 1024.  Parts of tiles with sinks are no longer than the longest
// other tile.
template <int A, int S>
Parts plan_parts(const AttnArgs& f, long ctas) {
  Parts p;
  p.ntiles = (f.Tk + A - 1) / A;
  p.nfirst = f.window ? (f.sinks + A - 1) / A : 0;
  if (p.nfirst > p.ntiles) p.nfirst = p.ntiles;
  long total = 0, mfirst = 0, mrest = 0;
  for (int t = 0; t < p.ntiles; ++t) {
    const long s = host_steps<A, S>(f, t);
    total += s;
    long& most = t < p.nfirst ? mfirst : mrest;
    if (s > most) most = s;
  }
  total *= (long)f.B * f.Hkv;
  long cap = total * 3 / (2 * ctas) + 1;
  if (cap < 4) cap = 4;
  if (cap > (1 << 28)) cap = 1 << 28;
  p.crest = (int)cap;
  p.cfirst = (int)(mrest >= 4 && mrest < cap ? mrest : cap);
  p.pfirst = (int)((mfirst + p.cfirst - 1) / p.cfirst);
  p.prest = (int)((mrest + cap - 1) / cap);
  if (p.pfirst < 1) p.pfirst = 1;
  if (p.prest < 1) p.prest = 1;
  return p;
}

// Workspace of the parts' sums (0 when no tile is cut).
inline size_t part_bytes(const AttnArgs& f, int A, const Parts& p) {
  if (!p.cut()) return 0;
  const size_t items = p.prest > 1 ? p.items() : (size_t)p.nfirst * p.pfirst;
  return items * f.B * f.Hkv * 2 * A * f.d * sizeof(float);
}

}  // namespace attn
}  // namespace gdr
