// Sliding-window attention and its gradients on the CUDA cores, all in fp32: fp32 tensors,
// and head size 32 (the tensor-core kernels are attn_tc_forward.cu, attn_tc_backward.cu).
// The mathematics and the mask are in attn_common.cuh.
//
// A CTA keeps a tile of 32 rows (queries, or for dk and dv keys) and streams tiles of 64 rows of
// the other side past it.  Two groups of 128 threads take the streamed tiles in turn, each with
// its own statistics and sums, which join at the end: one group alone leaves a warp for each
// scheduler, which issues a multiply-add every other cycle at best.  The threads of a group stand
// as 8 x 16, each with a 4 x 4 piece of the score tile and 4 rows x d/16 columns of the products
// over it.  One pass over the keys with the running maximum and sum; the backward rebuilds the
// probabilities from lse, once for dq and once for dk, dv (a CTA walks the query heads of its
// group itself, so no sum crosses CTAs and results are deterministic).
// Bound: fp32 multiply-adds, 4 d flops a pair forward, 14 d backward (two rebuilds).  777 tokens
// x 6 heads x 3 sequences (d = 64, forward + dk, dv + dq): tiles of 64 rows by 256 threads took
// 129 + 204 + 162 us, of 32 rows by one group 92 + 155 + 119.

#include "attn_parts.cuh"
#include "once.h"

namespace gdr {
namespace {

using namespace attn;

constexpr int kA = 32;          // rows of the tile that stays
constexpr int kB = 64;          // rows of the tiles that stream
constexpr int kGroup = 128;     // threads that share a streamed tile
constexpr int kThreads = 2 * kGroup;
constexpr int kLd = kB + 4;

__device__ __forceinline__ void group_sync(int g) {
  asm volatile("bar.sync %0, %1;" :: "r"(1 + g), "r"(kGroup) : "memory");
}

// rows r0 .. r0 + ROWS - 1 of x [rows][heads][D] into dst [ROWS][D + 4], zeros at and past `end`
// by the threads t of n
template <typename T, int D, int ROWS, int N>
__device__ __forceinline__ void load_tile(float* dst, const T* x, size_t row_stride, int r0,
                                          int end, int t) {
#pragma unroll 4
  for (int e = t; e < ROWS * (D / 4); e += N) {
    const int r = e / (D / 4), c = (e % (D / 4)) * 4;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < end) f = Elem<T>::load4(x + (size_t)(r0 + r) * row_stride + c);
    *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = f;
  }
}

// g[a][b] = sum_c x[4 ty + a][c] y[tx + 16 b][c], even and odd channels apart until the end
template <int D>
__device__ __forceinline__ void tile_dot(const float* x, const float* y, int ty, int tx,
                                         float (&g)[4][4]) {
  float2 s[4][4];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) s[a][b] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    float4 u[4], w[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      u[a] = *reinterpret_cast<const float4*>(x + (4 * ty + a) * (D + 4) + c);
      w[a] = *reinterpret_cast<const float4*>(y + (tx + 16 * a) * (D + 4) + c);
    }
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        s[a][b] = fma2(make_float2(u[a].x, u[a].y), make_float2(w[b].x, w[b].y), s[a][b]);
        s[a][b] = fma2(make_float2(u[a].z, u[a].w), make_float2(w[b].z, w[b].w), s[a][b]);
      }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) g[a][b] = s[a][b].x + s[a][b].y;
}

// The columns of thread tx: tx W + 16 W g + e, e < W, g < G; W consecutive ones per read.
template <int D>
struct Cols {
  static constexpr int N = D / 16, W = N < 4 ? N : 4, G = N / W;
  static __device__ __forceinline__ void load(const float* row, int tx, float (&v)[N]) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float* p = row + tx * W + 16 * W * g;
      if constexpr (W == 4) {
        const float4 f = *reinterpret_cast<const float4*>(p);
        v[4 * g] = f.x, v[4 * g + 1] = f.y, v[4 * g + 2] = f.z, v[4 * g + 3] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(p);
        v[0] = f.x, v[1] = f.y;
      }
    }
  }
};

// acc[a][..] += sum_j m[4 ty + a][j] y[j][columns of tx]
template <int D>
__device__ __forceinline__ void tile_acc(const float* m, const float* y, int ty, int tx,
                                         float (&acc)[4][Cols<D>::N]) {
  using C = Cols<D>;
#pragma unroll 2
  for (int j = 0; j < kB; j += 4) {
    float p[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float4 f = *reinterpret_cast<const float4*>(m + (4 * ty + a) * kLd + j);
      p[a][0] = f.x, p[a][1] = f.y, p[a][2] = f.z, p[a][3] = f.w;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float v[C::N];
      C::load(y + (j + u) * (D + 4), tx, v);
#pragma unroll
      for (int e = 0; e < C::N; ++e)
#pragma unroll
        for (int a = 0; a < 4; ++a) acc[a][e] = fmaf(p[a][u], v[e], acc[a][e]);
    }
  }
}
template <typename T, int D>
__device__ __forceinline__ void store_rows(T* x, size_t row_stride, int r0, int end, int ty,
                                           int tx, const float (&acc)[4][Cols<D>::N]) {
  using C = Cols<D>;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int r = r0 + 4 * ty + a;
    if (r < end) {
#pragma unroll
      for (int g = 0; g < C::G; ++g)
#pragma unroll
        for (int e = 0; e < C::W; ++e)
          Elem<T>::store(x + (size_t)r * row_stride + tx * C::W + 16 * C::W * g + e,
                         acc[a][g * C::W + e]);
    }
  }
}

// a part's sums as part_at places them
template <int D>
__device__ __forceinline__ void store_part(float* x, int ty, int tx,
                                           const float (&acc)[4][Cols<D>::N]) {
  using C = Cols<D>;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int g = 0; g < C::G; ++g)
#pragma unroll
      for (int e = 0; e < C::W; ++e) {
        const int c = tx * C::W + 16 * C::W * g + e;
        x[((c >> 3) * kA + 4 * ty + a) * 8 + (c & 7)] = acc[a][g * C::W + e];
      }
}

__device__ __forceinline__ float row_max(float x) {   // over the 16 lanes of a tile row
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int D>
struct FwdSmem {
  float q[kA * (D + 4)];
  struct {
    float k[kB * (D + 4)], v[kB * (D + 4)], p[kA * kLd];
  } g[2];
  float mx[kA], sum[kA];            // the second group's, for the join
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
attn_forward_simt(const AttnArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  FwdSmem<D>& sm = *reinterpret_cast<FwdSmem<D>*>(smem_raw);
  const int nq = (a.Tq + kA - 1) / kA;
  // the last queries see the most keys without a window, so they start first
  const int bh = blockIdx.x % (a.B * a.Hq), h = bh % a.Hq, b = bh / a.Hq;
  const int i0 = (nq - 1 - (int)(blockIdx.x / (unsigned)(a.B * a.Hq))) * kA;
  const int hk = h / (a.Hq / a.Hkv);
  const int grp = threadIdx.x / kGroup, tid = threadIdx.x % kGroup, ty = tid >> 4, tx = tid & 15;
  const Mask m = make_mask(a.lengths, b, a.Tq, a.Tk, a.window, a.sinks);
  const KeyTiles kt = key_tiles<kB>(m, i0, min(i0 + kA, a.Tq) - 1);
  const size_t qs = (size_t)a.Hq * D, ks = (size_t)a.Hkv * D;
  const T* q = (const T*)a.q + (size_t)b * a.Tq * qs + (size_t)h * D;
  const T* k = (const T*)a.k + (size_t)b * a.Tk * ks + (size_t)hk * D;
  const T* v = (const T*)a.v + (size_t)b * a.Tk * ks + (size_t)hk * D;
  load_tile<T, D, kA, kThreads>(sm.q, q, qs, i0, a.Tq, threadIdx.x);
  __syncthreads();
  auto& st = sm.g[grp];
  float acc[4][Cols<D>::N] = {};
  float mx[4], sum[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) mx[r] = -INFINITY, sum[r] = 0.f;
  const float c = a.scale * kLog2e;
  for (int x = grp; x < kt.count(); x += 2) {
    const int j0 = kt.tile(x) * kB;
    group_sync(grp);
    load_tile<T, D, kB, kGroup>(st.k, k, ks, j0, m.len, tid);
    load_tile<T, D, kB, kGroup>(st.v, v, ks, j0, m.len, tid);
    group_sync(grp);
    float g[4][4];
    tile_dot<D>(sm.q, st.k, ty, tx, g);
    const bool whole = all_visible(m, m.off + i0, m.off + i0 + kA - 1, j0, j0 + kB - 1);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float top = -INFINITY;
      const RowCols rc = row_cols(m, m.off + i0 + 4 * ty + r, j0);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[r][e] = whole | rc.sees(tx + 16 * e) ? g[r][e] * c : -INFINITY;
        top = fmaxf(top, g[r][e]);
      }
      const float now = fmaxf(mx[r], row_max(top));
      const float base = now == -INFINITY ? 0.f : now;
      const float f = ex2(mx[r] - base);
      mx[r] = now;
      float part = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = ex2(g[r][e] - base);
        st.p[(4 * ty + r) * kLd + tx + 16 * e] = w;
        part += w;
      }
      sum[r] = fmaf(sum[r], f, part);       // this thread's columns only, until the end
#pragma unroll
      for (int e = 0; e < Cols<D>::N; ++e) acc[r][e] *= f;
    }
    __syncwarp();       // a tile row's 16 lanes lie in one warp
    tile_acc<D>(st.p, st.v, ty, tx, acc);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) sum[r] = row_sum(sum[r]);
  // the second group hands over its rows (in its key buffer), the first adds and writes them
  float* other = sm.g[1].k;
  if (grp == 1) {
    group_sync(1);            // all of it is done with the buffer
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (tx == 0) sm.mx[4 * ty + r] = mx[r], sm.sum[4 * ty + r] = sum[r];
#pragma unroll
      for (int e = 0; e < Cols<D>::N; ++e)
        other[((4 * ty + r) * Cols<D>::N + e) * 16 + tx] = acc[r][e];
    }
  }
  __syncthreads();
  if (grp == 1) return;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + 4 * ty + r;
    const float m2 = sm.mx[4 * ty + r], now = fmaxf(mx[r], m2);
    const float base = now == -INFINITY ? 0.f : now;
    const float f1 = ex2(mx[r] - base), f2 = ex2(m2 - base);
    mx[r] = now;
    sum[r] = fmaf(sum[r], f1, sm.sum[4 * ty + r] * f2);
#pragma unroll
    for (int e = 0; e < Cols<D>::N; ++e)
      acc[r][e] = fmaf(acc[r][e], f1, other[((4 * ty + r) * Cols<D>::N + e) * 16 + tx] * f2);
    const float inv = sum[r] == 0.f ? 0.f : 1.f / sum[r];
#pragma unroll
    for (int e = 0; e < Cols<D>::N; ++e) acc[r][e] *= inv;
    if (tx == 0 && i < a.Tq && a.lse)
      a.lse[((size_t)b * a.Hq + h) * a.Tq + i] =
          mx[r] == -INFINITY ? -INFINITY : (mx[r] + log2f(sum[r])) * kLn2;
  }
  store_rows<T, D>((T*)a.o + (size_t)b * a.Tq * qs + (size_t)h * D, qs, i0, a.Tq, ty, tx, acc);
}

template <int D>
struct DqSmem {
  float q[kA * (D + 4)], d[kA * (D + 4)];
  struct {
    float k[kB * (D + 4)], v[kB * (D + 4)], s[kA * kLd];
  } g[2];
};

// The second group's sums to the first, through `buf`.  Returns whether this is the first.
template <int N>
__device__ __forceinline__ bool join_groups(float* buf, int grp, int ty, int tx,
                                            float (&acc)[4][N]) {
  __syncthreads();
  if (grp == 1) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int e = 0; e < N; ++e) buf[((4 * ty + r) * N + e) * 16 + tx] = acc[r][e];
  }
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int e = 0; e < N; ++e) acc[r][e] += buf[((4 * ty + r) * N + e) * 16 + tx];
  }
  return grp == 0;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
attn_dq_simt(const AttnGradArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  DqSmem<D>& sm = *reinterpret_cast<DqSmem<D>*>(smem_raw);
  const AttnArgs& f = a.f;
  const int nq = (f.Tq + kA - 1) / kA;
  const int bh = blockIdx.x % (f.B * f.Hq), h = bh % f.Hq, b = bh / f.Hq;
  const int i0 = (nq - 1 - (int)(blockIdx.x / (unsigned)(f.B * f.Hq))) * kA;
  const int hk = h / (f.Hq / f.Hkv);
  const int grp = threadIdx.x / kGroup, tid = threadIdx.x % kGroup, ty = tid >> 4, tx = tid & 15;
  const Mask m = make_mask(f.lengths, b, f.Tq, f.Tk, f.window, f.sinks);
  const KeyTiles kt = key_tiles<kB>(m, i0, min(i0 + kA, f.Tq) - 1);
  const size_t qs = (size_t)f.Hq * D, ks = (size_t)f.Hkv * D;
  const size_t qat = (size_t)b * f.Tq * qs + (size_t)h * D;
  const size_t kat = (size_t)b * f.Tk * ks + (size_t)hk * D;
  // rows past the length see nothing; their q and do may hold anything
  const int end = min(f.Tq, m.len - m.off);
  load_tile<T, D, kA, kThreads>(sm.q, (const T*)f.q + qat, qs, i0, end, threadIdx.x);
  load_tile<T, D, kA, kThreads>(sm.d, (const T*)a.dO + qat, qs, i0, end, threadIdx.x);
  __syncthreads();
  auto& st = sm.g[grp];
  float lse[4], delta[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + 4 * ty + r;
    const size_t at = ((size_t)b * f.Hq + h) * f.Tq + i;
    lse[r] = i < end ? f.lse[at] : 0.f;
    delta[r] = i < end ? a.delta[at] : 0.f;
  }
  float acc[4][Cols<D>::N] = {};
  for (int x = grp; x < kt.count(); x += 2) {
    const int j0 = kt.tile(x) * kB;
    group_sync(grp);
    load_tile<T, D, kB, kGroup>(st.k, (const T*)f.k + kat, ks, j0, m.len, tid);
    load_tile<T, D, kB, kGroup>(st.v, (const T*)f.v + kat, ks, j0, m.len, tid);
    group_sync(grp);
    float g[4][4], dp[4][4];
    tile_dot<D>(sm.q, st.k, ty, tx, g);
    tile_dot<D>(sm.d, st.v, ty, tx, dp);
    const bool whole = all_visible(m, m.off + i0, m.off + i0 + kA - 1, j0, j0 + kB - 1);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const RowCols rc = row_cols(m, m.off + i0 + 4 * ty + r, j0);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = tx + 16 * e;
        const float w = ex2((g[r][e] * f.scale - lse[r]) * kLog2e);
        st.s[(4 * ty + r) * kLd + j] =
            whole | rc.sees(j) ? f.scale * w * (dp[r][e] - delta[r]) : 0.f;
      }
    }
    __syncwarp();
    tile_acc<D>(st.s, st.k, ty, tx, acc);
  }
  if (join_groups(sm.g[1].k, grp, ty, tx, acc))
    store_rows<T, D>((T*)a.dq + qat, qs, i0, f.Tq, ty, tx, acc);
}

template <int D>
struct DkvSmem {
  float k[kA * (D + 4)], v[kA * (D + 4)];
  struct {
    float q[kB * (D + 4)], d[kB * (D + 4)];
    float p[kA * kLd], s[kA * kLd];
    float lse[kB], delta[kB];
  } g[2];
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
attn_dkv_simt(const AttnGradArgs a, const Parts parts) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  DkvSmem<D>& sm = *reinterpret_cast<DkvSmem<D>*>(smem_raw);
  const AttnArgs& f = a.f;
  // the first keys, which the most queries see without a window, start first
  const int bh = blockIdx.x % (f.B * f.Hkv), hk = bh % f.Hkv, b = bh / f.Hkv;
  const int item = blockIdx.x / (unsigned)(f.B * f.Hkv);
  int tile, part;
  parts.locate(item, tile, part);
  const int j0 = tile * kA;
  const int G = f.Hq / f.Hkv;
  const int grp = threadIdx.x / kGroup, tid = threadIdx.x % kGroup, ty = tid >> 4, tx = tid & 15;
  const Mask m = make_mask(f.lengths, b, f.Tq, f.Tk, f.window, f.sinks);
  int first, nt;
  tile_steps<kA, kB>(m, j0, f.Tk, f.Tq, first, nt);
  const int used = parts.used(G * nt, tile);
  if (part >= used) return;
  const int per = (G * nt + used - 1) / used, x1 = min(G * nt, (part + 1) * per);
  const size_t qs = (size_t)f.Hq * D, ks = (size_t)f.Hkv * D;
  const size_t kat = (size_t)b * f.Tk * ks + (size_t)hk * D;
  load_tile<T, D, kA, kThreads>(sm.k, (const T*)f.k + kat, ks, j0, m.len, threadIdx.x);
  load_tile<T, D, kA, kThreads>(sm.v, (const T*)f.v + kat, ks, j0, m.len, threadIdx.x);
  __syncthreads();
  auto& st = sm.g[grp];
  const int end = min(f.Tq, m.len - m.off);
  float dk[4][Cols<D>::N] = {}, dv[4][Cols<D>::N] = {};
  for (int x = part * per + grp; x < x1; x += 2) {
    const int h = hk * G + x / nt, i0 = (first + x % nt) * kB;
    const size_t qat = (size_t)b * f.Tq * qs + (size_t)h * D;
    group_sync(grp);
    load_tile<T, D, kB, kGroup>(st.q, (const T*)f.q + qat, qs, i0, end, tid);
    load_tile<T, D, kB, kGroup>(st.d, (const T*)a.dO + qat, qs, i0, end, tid);
    if (tid < kB) {
      const size_t at = ((size_t)b * f.Hq + h) * f.Tq + i0 + tid;
      st.lse[tid] = i0 + tid < end ? f.lse[at] : 0.f;
      st.delta[tid] = i0 + tid < end ? a.delta[at] : 0.f;
    }
    group_sync(grp);
    float g[4][4], dp[4][4];
    tile_dot<D>(sm.k, st.q, ty, tx, g);
    tile_dot<D>(sm.v, st.d, ty, tx, dp);
    const int p0 = m.off + i0;
    const bool whole = all_visible(m, p0, p0 + kB - 1, j0, j0 + kA - 1);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const RowCols rc = col_rows(m, j0 + 4 * ty + r, p0);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = tx + 16 * e, at = (4 * ty + r) * kLd + i;
        const bool sees = whole | rc.sees(i);
        const float w = sees ? ex2((g[r][e] * f.scale - st.lse[i]) * kLog2e) : 0.f;
        st.p[at] = w;
        st.s[at] = sees ? f.scale * w * (dp[r][e] - st.delta[i]) : 0.f;
      }
    }
    __syncwarp();
    tile_acc<D>(st.p, st.d, ty, tx, dv);
    tile_acc<D>(st.s, st.q, ty, tx, dk);
  }
  const bool mine = join_groups(sm.g[1].q, grp, ty, tx, dk);
  join_groups(sm.g[1].d, grp, ty, tx, dv);
  if (mine && used > 1) {
    float* pv = a.part + part_at(f, kA, D, item, bh, 0, 0, 0);
    store_part<D>(pv, ty, tx, dv);
    store_part<D>(pv + kA * D, ty, tx, dk);
  } else if (mine) {
    store_rows<T, D>((T*)a.dk + kat, ks, j0, f.Tk, ty, tx, dk);
    store_rows<T, D>((T*)a.dv + kat, ks, j0, f.Tk, ty, tx, dv);
  }
}

// D_i = do_i . o_i: 16 bytes of both rows a thread, four rows in flight.
template <typename T, int D>
__global__ void __launch_bounds__(256)
attn_delta_kernel(const T* __restrict__ o, const T* __restrict__ dO, float* __restrict__ delta,
                  int B, int Tq, int Hq) {
  constexpr int PER = 16 / sizeof(T), LPR = D / PER;      // elements a thread, lanes a row
  constexpr int ROWS = 256 / LPR, R = 4;
  const size_t rows = (size_t)B * Tq * Hq;                // (b, i, h)
  const size_t first = (size_t)blockIdx.x * ROWS * R + threadIdx.x / LPR;
  const int c = threadIdx.x % LPR * PER;
  float s[R];
  float4 x[R][PER / 4], y[R][PER / 4];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const size_t row = min(first + (size_t)r * ROWS, rows - 1);
#pragma unroll
    for (int e = 0; e < PER / 4; ++e) {
      x[r][e] = Elem<T>::load4(o + row * D + c + 4 * e);
      y[r][e] = Elem<T>::load4(dO + row * D + c + 4 * e);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    s[r] = 0.f;
#pragma unroll
    for (int e = 0; e < PER / 4; ++e)
      s[r] = fmaf(x[r][e].x, y[r][e].x,
                  fmaf(x[r][e].y, y[r][e].y,
                       fmaf(x[r][e].z, y[r][e].z, fmaf(x[r][e].w, y[r][e].w, s[r]))));
#pragma unroll
    for (int f = LPR / 2; f; f >>= 1) s[r] += __shfl_xor_sync(0xffffffffu, s[r], f);
    const size_t row = first + (size_t)r * ROWS;
    if (row < rows && c == 0) {
      const size_t h = row % Hq, bi = row / Hq;
      delta[((bi / Tq) * Hq + h) * Tq + bi % Tq] = s[r];
    }
  }
}

// Queries without any key: lse = -inf (and o = 0).
__global__ void __launch_bounds__(256) attn_no_keys_kernel(float* lse, size_t n) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) lse[i] = -INFINITY;
}

template <typename T, int D>
cudaError_t forward_t(const AttnArgs& a, cudaStream_t st) {
  auto kern = attn_forward_simt<T, D>;
  constexpr int smem = (int)sizeof(FwdSmem<D>);
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)((a.Tq + kA - 1) / kA) * (unsigned)(a.Hq * a.B), kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t delta_t(const AttnGradArgs& a, cudaStream_t st) {
  const size_t rows = (size_t)a.f.B * a.f.Tq * a.f.Hq;
  constexpr size_t per = 4 * (256 / (D * sizeof(T) / 16));
  attn_delta_kernel<T, D><<<(unsigned)((rows + per - 1) / per), 256, 0, st>>>(
      (const T*)a.f.o, (const T*)a.dO, a.delta, a.f.B, a.f.Tq, a.f.Hq);
  return cudaGetLastError();
}

// Two places on an SM.  attn_dkv_simt has two CTAs there at d = 32 (80 KB of shared memory each) but
// one at 64 and 128 (120 and 200 KB), so there a part is at most three quarters of an SM's mean
// share instead of one and a half.  That measured better on the whole than counting one (forward
// and gradients, fp32): 2 x 600 tokens, 16 heads of 64 to 2, window 200: 192 us against 228; 1024
// tokens, 8 heads of 128 to 2: 416 against 400; 1500 tokens, 4 heads of 64, and 3 x 777, 6 heads of
// 64: equal.
Parts plan_simt(const AttnArgs& f) { return plan_parts<kA, kB>(f, 2 * 148); }

template <typename T, int D>
cudaError_t backward_t(const AttnGradArgs& a, cudaStream_t st) {
  auto kq = attn_dq_simt<T, D>;
  auto kk = attn_dkv_simt<T, D>;
  constexpr int sq = (int)sizeof(DqSmem<D>), sk = (int)sizeof(DkvSmem<D>);
  static std::atomic<unsigned long long> done{0}, done2{0};
  cudaError_t e = allow_smem(kq, sq, done);
  if (e == cudaSuccess)
    e = allow_smem(kk, sk, done2);
  if (e != cudaSuccess) return e;
  const Parts p = plan_simt(a.f);
  kk<<<(unsigned)p.items() * (unsigned)(a.f.Hkv * a.f.B), kThreads, sk, st>>>(a, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = launch_dkv_join<T, D, kA, kB>(a, p, st)) != cudaSuccess) return e;
  kq<<<(unsigned)((a.f.Tq + kA - 1) / kA) * (unsigned)(a.f.Hq * a.f.B), kThreads, sq, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

// bf16 with d = 64 or 128 runs on the tensor cores, all but do . o.
#define GDR_BY_TYPE(fn, dtype, d, ...)                                              \
  do {                                                                              \
    if ((dtype) == GDR_F32) {                                                       \
      if ((d) == 32) return fn<float, 32>(__VA_ARGS__);                             \
      if ((d) == 64) return fn<float, 64>(__VA_ARGS__);                             \
      if ((d) == 128) return fn<float, 128>(__VA_ARGS__);                           \
    } else if ((d) == 32) {                                                         \
      return fn<__nv_bfloat16, 32>(__VA_ARGS__);                                    \
    }                                                                               \
  } while (0)

size_t attn_backward_simt_bytes(const AttnArgs& f) { return part_bytes(f, kA, plan_simt(f)); }
cudaError_t launch_attn_forward_simt(const AttnArgs& a, cudaStream_t st) {
  GDR_BY_TYPE(forward_t, a.dtype, a.d, a, st);
  return cudaErrorInvalidValue;
}
cudaError_t launch_attn_delta(const AttnGradArgs& a, cudaStream_t st) {
  GDR_BY_TYPE(delta_t, a.f.dtype, a.f.d, a, st);
  return a.f.d == 64 ? delta_t<__nv_bfloat16, 64>(a, st) : delta_t<__nv_bfloat16, 128>(a, st);
}
cudaError_t launch_attn_backward_simt(const AttnGradArgs& a, cudaStream_t st) {
  GDR_BY_TYPE(backward_t, a.f.dtype, a.f.d, a, st);
  return cudaErrorInvalidValue;
}
cudaError_t launch_attn_no_keys(const AttnArgs& a, cudaStream_t st) {
  const size_t rows = (size_t)a.B * a.Tq * a.Hq, e = a.dtype == GDR_F32 ? 4 : 2;
  cudaError_t r = cudaMemsetAsync(a.o, 0, rows * a.d * e, st);
  if (r != cudaSuccess || !a.lse) return r;
  attn_no_keys_kernel<<<(unsigned)((rows + 255) / 256), 256, 0, st>>>(a.lse, rows);
  return cudaGetLastError();
}

}  // namespace gdr
