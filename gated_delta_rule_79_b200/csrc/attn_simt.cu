// Sliding-window attention and its gradients on the CUDA cores, all in fp32: fp32 tensors,
// and head size 32 (the tensor-core kernels are attn_tc_forward.cu, attn_tc_backward.cu).
// The mathematics and the mask are in attn_common.cuh.
//
// Tiles of 64 queries x 64 keys, 256 threads as 16 x 16, each with a 4 x 4 piece of the
// score tile and 4 rows x d/16 columns of the products over it.  One pass over the keys
// with the running maximum and sum; the backward rebuilds the probabilities from lse, once
// for dq (a CTA per query tile) and once for dk, dv (a CTA per key tile, which walks the
// query heads of its group itself, so no sum crosses CTAs and results are deterministic).
// Bound: fp32 multiply-adds, 4 d flops a pair forward, 14 d backward (two rebuilds).

#include "attn_common.cuh"
#include "once.h"

namespace gdr {
namespace {

using namespace attn;

constexpr int kB = 64;          // queries and keys of a tile
constexpr int kThreads = 256;
constexpr int kLd = kB + 4;

// rows r0 .. r0 + 63 of x [rows][heads][D] into dst [64][D + 4], zeros at and past `end`
template <typename T, int D>
__device__ __forceinline__ void load_tile(float* dst, const T* x, size_t row_stride, int r0,
                                          int end) {
  for (int e = threadIdx.x; e < kB * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c = (e % (D / 4)) * 4;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < end) f = Elem<T>::load4(x + (size_t)(r0 + r) * row_stride + c);
    *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = f;
  }
}

// g[a][b] = sum_c x[4 ty + a][c] y[tx + 16 b][c]
template <int D>
__device__ __forceinline__ void tile_dot(const float* x, const float* y, int ty, int tx,
                                         float (&g)[4][4]) {
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) g[a][b] = 0.f;
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
      for (int b = 0; b < 4; ++b)
        g[a][b] = fmaf(u[a].x, w[b].x,
                       fmaf(u[a].y, w[b].y, fmaf(u[a].z, w[b].z, fmaf(u[a].w, w[b].w, g[a][b]))));
  }
}

// acc[a][..] += sum_j m[4 ty + a][j] y[j][columns of tx]  (columns tx*W + 16*W*g + e)
template <int D>
struct Cols {
  static constexpr int N = D / 16, W = N < 4 ? N : 4, G = N / W;
};
template <int D>
__device__ __forceinline__ void tile_acc(const float* m, const float* y, int ty, int tx,
                                         float (&acc)[4][Cols<D>::N]) {
  using C = Cols<D>;
#pragma unroll 4
  for (int j = 0; j < kB; ++j) {
    float p[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) p[a] = m[(4 * ty + a) * kLd + j];
#pragma unroll
    for (int g = 0; g < C::G; ++g)
#pragma unroll
      for (int e = 0; e < C::W; ++e) {
        const float s = y[j * (D + 4) + tx * C::W + 16 * C::W * g + e];
#pragma unroll
        for (int a = 0; a < 4; ++a) acc[a][g * C::W + e] = fmaf(p[a], s, acc[a][g * C::W + e]);
      }
  }
}
// the same with m transposed: acc[a][..] += sum_i m[i][4 ty + a] y[i][..]
template <int D>
__device__ __forceinline__ void tile_acc_t(const float* m, const float* y, int ty, int tx,
                                           float (&acc)[4][Cols<D>::N]) {
  using C = Cols<D>;
#pragma unroll 4
  for (int i = 0; i < kB; ++i) {
    const float4 p4 = *reinterpret_cast<const float4*>(m + i * kLd + 4 * ty);
    const float p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
    for (int g = 0; g < C::G; ++g)
#pragma unroll
      for (int e = 0; e < C::W; ++e) {
        const float s = y[i * (D + 4) + tx * C::W + 16 * C::W * g + e];
#pragma unroll
        for (int a = 0; a < 4; ++a) acc[a][g * C::W + e] = fmaf(p[a], s, acc[a][g * C::W + e]);
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
  float q[kB * (D + 4)], k[kB * (D + 4)], v[kB * (D + 4)], p[kB * kLd];
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
attn_forward_simt(const AttnArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  FwdSmem<D>& sm = *reinterpret_cast<FwdSmem<D>*>(smem_raw);
  const int nq = (a.Tq + kB - 1) / kB;
  // the last query tiles see the most keys without a window, so they start first
  const int qt = nq - 1 - (int)(blockIdx.x % nq);
  const int bh = blockIdx.x / nq, h = bh % a.Hq, b = bh / a.Hq;
  const int hk = h / (a.Hq / a.Hkv);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int i0 = qt * kB;
  const Mask m = make_mask(a.lengths, b, a.Tq, a.Tk, a.window, a.sinks);
  const KeyTiles kt = key_tiles<kB>(m, i0, min(i0 + kB, a.Tq) - 1);
  const size_t qs = (size_t)a.Hq * D, ks = (size_t)a.Hkv * D;
  const T* q = (const T*)a.q + (size_t)b * a.Tq * qs + (size_t)h * D;
  const T* k = (const T*)a.k + (size_t)b * a.Tk * ks + (size_t)hk * D;
  const T* v = (const T*)a.v + (size_t)b * a.Tk * ks + (size_t)hk * D;
  load_tile<T, D>(sm.q, q, qs, i0, a.Tq);
  float acc[4][Cols<D>::N] = {};
  float mx[4], sum[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) mx[r] = -INFINITY, sum[r] = 0.f;
  const float c = a.scale * kLog2e;
  for (int x = 0; x < kt.count(); ++x) {
    const int j0 = kt.tile(x) * kB;
    __syncthreads();
    load_tile<T, D>(sm.k, k, ks, j0, m.len);
    load_tile<T, D>(sm.v, v, ks, j0, m.len);
    __syncthreads();
    float g[4][4];
    tile_dot<D>(sm.q, sm.k, ty, tx, g);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int pos = m.off + i0 + 4 * ty + r;
      float top = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[r][e] = m.sees(pos, j0 + tx + 16 * e) ? g[r][e] * c : -INFINITY;
        top = fmaxf(top, g[r][e]);
      }
      const float now = fmaxf(mx[r], row_max(top));
      const float base = now == -INFINITY ? 0.f : now;
      const float f = exp2f(mx[r] - base);
      mx[r] = now;
      float part = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = exp2f(g[r][e] - base);
        sm.p[(4 * ty + r) * kLd + tx + 16 * e] = w;
        part += w;
      }
      sum[r] = fmaf(sum[r], f, row_sum(part));
#pragma unroll
      for (int e = 0; e < Cols<D>::N; ++e) acc[r][e] *= f;
    }
    __syncwarp();       // a tile row's 16 lanes lie in one warp
    tile_acc<D>(sm.p, sm.v, ty, tx, acc);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + 4 * ty + r;
    const float inv = sum[r] > 0.f || sum[r] != sum[r] ? 1.f / sum[r] : 0.f;
#pragma unroll
    for (int e = 0; e < Cols<D>::N; ++e) acc[r][e] *= inv;
    if (tx == 0 && i < a.Tq && a.lse)
      a.lse[((size_t)b * a.Hq + h) * a.Tq + i] =
          mx[r] == -INFINITY ? -INFINITY : (mx[r] + log2f(sum[r])) * kLn2;
  }
  store_rows<T, D>((T*)a.o + (size_t)b * a.Tq * qs + (size_t)h * D, qs, i0, a.Tq, ty, tx, acc);
}

template <int D>
struct BwdSmem {
  float q[kB * (D + 4)], k[kB * (D + 4)], v[kB * (D + 4)], d[kB * (D + 4)];
  float p[kB * kLd], s[kB * kLd];
  float lse[kB], delta[kB];
};

// The tile's probabilities (into sm.p when wanted) and score gradients (into sm.s), from
// the loaded q, k, v, do, lse, delta tiles.
template <int D, bool KEEP_P>
__device__ __forceinline__ void tile_grads(BwdSmem<D>& sm, const Mask& m, int i0, int j0,
                                           float scale, int ty, int tx) {
  float g[4][4], dp[4][4];
  tile_dot<D>(sm.q, sm.k, ty, tx, g);
  tile_dot<D>(sm.d, sm.v, ty, tx, dp);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = 4 * ty + r, pos = m.off + i0 + i;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = tx + 16 * e;
      const bool sees = m.sees(pos, j0 + j);
      const float w = sees ? exp2f((g[r][e] * scale - sm.lse[i]) * kLog2e) : 0.f;
      if (KEEP_P) sm.p[i * kLd + j] = w;
      sm.s[i * kLd + j] = sees ? scale * w * (dp[r][e] - sm.delta[i]) : 0.f;
    }
  }
}

template <typename T, int D>
__device__ __forceinline__ void load_query_side(BwdSmem<D>& sm, const AttnGradArgs& a, int b,
                                                int h, int i0, int end) {
  const size_t qs = (size_t)a.f.Hq * D;
  const size_t at = (size_t)b * a.f.Tq * qs + (size_t)h * D;
  load_tile<T, D>(sm.q, (const T*)a.f.q + at, qs, i0, end);
  load_tile<T, D>(sm.d, (const T*)a.dO + at, qs, i0, end);
  if (threadIdx.x < kB) {
    const int i = i0 + threadIdx.x;
    const size_t r = ((size_t)b * a.f.Hq + h) * a.f.Tq + i;
    sm.lse[threadIdx.x] = i < end ? a.f.lse[r] : 0.f;
    sm.delta[threadIdx.x] = i < end ? a.delta[r] : 0.f;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
attn_dq_simt(const AttnGradArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  BwdSmem<D>& sm = *reinterpret_cast<BwdSmem<D>*>(smem_raw);
  const int nq = (a.f.Tq + kB - 1) / kB;
  const int qt = nq - 1 - (int)(blockIdx.x % nq);
  const int bh = blockIdx.x / nq, h = bh % a.f.Hq, b = bh / a.f.Hq;
  const int hk = h / (a.f.Hq / a.f.Hkv);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int i0 = qt * kB;
  const Mask m = make_mask(a.f.lengths, b, a.f.Tq, a.f.Tk, a.f.window, a.f.sinks);
  const KeyTiles kt = key_tiles<kB>(m, i0, min(i0 + kB, a.f.Tq) - 1);
  const size_t qs = (size_t)a.f.Hq * D, ks = (size_t)a.f.Hkv * D;
  const size_t kat = (size_t)b * a.f.Tk * ks + (size_t)hk * D;
  // rows past the length see nothing; their q and do may hold anything
  load_query_side<T, D>(sm, a, b, h, i0, min(a.f.Tq, m.len - m.off));
  float acc[4][Cols<D>::N] = {};
  for (int x = 0; x < kt.count(); ++x) {
    const int j0 = kt.tile(x) * kB;
    __syncthreads();
    load_tile<T, D>(sm.k, (const T*)a.f.k + kat, ks, j0, m.len);
    load_tile<T, D>(sm.v, (const T*)a.f.v + kat, ks, j0, m.len);
    __syncthreads();
    tile_grads<D, false>(sm, m, i0, j0, a.f.scale, ty, tx);
    __syncwarp();
    tile_acc<D>(sm.s, sm.k, ty, tx, acc);
  }
  store_rows<T, D>((T*)a.dq + (size_t)b * a.f.Tq * qs + (size_t)h * D, qs, i0, a.f.Tq, ty, tx,
                   acc);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
attn_dkv_simt(const AttnGradArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  BwdSmem<D>& sm = *reinterpret_cast<BwdSmem<D>*>(smem_raw);
  const int nk = (a.f.Tk + kB - 1) / kB;
  const int kt = blockIdx.x % nk;
  const int bh = blockIdx.x / nk, hk = bh % a.f.Hkv, b = bh / a.f.Hkv;
  const int G = a.f.Hq / a.f.Hkv;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int j0 = kt * kB;
  const Mask m = make_mask(a.f.lengths, b, a.f.Tq, a.f.Tk, a.f.window, a.f.sinks);
  const size_t ks = (size_t)a.f.Hkv * D;
  const size_t kat = (size_t)b * a.f.Tk * ks + (size_t)hk * D;
  load_tile<T, D>(sm.k, (const T*)a.f.k + kat, ks, j0, m.len);
  load_tile<T, D>(sm.v, (const T*)a.f.v + kat, ks, j0, m.len);
  int lo, hi;
  query_range(m, j0, min(j0 + kB, a.f.Tk) - 1, a.f.Tq, lo, hi);
  float dk[4][Cols<D>::N] = {}, dv[4][Cols<D>::N] = {};
  for (int g = 0; g < G; ++g)
    for (int i0 = lo / kB * kB; i0 < hi; i0 += kB) {
      __syncthreads();
      load_query_side<T, D>(sm, a, b, hk * G + g, i0, min(a.f.Tq, m.len - m.off));
      __syncthreads();
      tile_grads<D, true>(sm, m, i0, j0, a.f.scale, ty, tx);
      __syncthreads();
      tile_acc_t<D>(sm.p, sm.d, ty, tx, dv);
      tile_acc_t<D>(sm.s, sm.q, ty, tx, dk);
    }
  store_rows<T, D>((T*)a.dk + kat, ks, j0, a.f.Tk, ty, tx, dk);
  store_rows<T, D>((T*)a.dv + kat, ks, j0, a.f.Tk, ty, tx, dv);
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

template <typename T, int D>
cudaError_t forward_t(const AttnArgs& a, cudaStream_t st) {
  auto kern = attn_forward_simt<T, D>;
  constexpr int smem = (int)sizeof(FwdSmem<D>);
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)((a.Tq + kB - 1) / kB * a.Hq * a.B), kThreads, smem, st>>>(a);
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

template <typename T, int D>
cudaError_t backward_t(const AttnGradArgs& a, cudaStream_t st) {
  constexpr int smem = (int)sizeof(BwdSmem<D>);
  auto kq = attn_dq_simt<T, D>;
  auto kk = attn_dkv_simt<T, D>;
  static std::atomic<unsigned long long> done{0}, done2{0};
  cudaError_t e = allow_smem(kq, smem, done);
  if (e == cudaSuccess)
    e = allow_smem(kk, smem, done2);
  if (e != cudaSuccess) return e;
  if (a.f.Tq > 0) {
    kq<<<(unsigned)((a.f.Tq + kB - 1) / kB * a.f.Hq * a.f.B), kThreads, smem, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  kk<<<(unsigned)((a.f.Tk + kB - 1) / kB * a.f.Hkv * a.f.B), kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

#define GDR_BY_TYPE(fn, dtype, d, ...)                                              \
  do {                                                                              \
    if ((dtype) == GDR_F32) {                                                       \
      if ((d) == 32) return fn<float, 32>(__VA_ARGS__);                             \
      if ((d) == 64) return fn<float, 64>(__VA_ARGS__);                             \
      if ((d) == 128) return fn<float, 128>(__VA_ARGS__);                           \
    } else {                                                                        \
      if ((d) == 32) return fn<__nv_bfloat16, 32>(__VA_ARGS__);                     \
      if ((d) == 64) return fn<__nv_bfloat16, 64>(__VA_ARGS__);                     \
      if ((d) == 128) return fn<__nv_bfloat16, 128>(__VA_ARGS__);                   \
    }                                                                               \
    return cudaErrorInvalidValue;                                                   \
  } while (0)

cudaError_t launch_attn_forward_simt(const AttnArgs& a, cudaStream_t st) {
  GDR_BY_TYPE(forward_t, a.dtype, a.d, a, st);
}
cudaError_t launch_attn_delta(const AttnGradArgs& a, cudaStream_t st) {
  GDR_BY_TYPE(delta_t, a.f.dtype, a.f.d, a, st);
}
cudaError_t launch_attn_backward_simt(const AttnGradArgs& a, cudaStream_t st) {
  GDR_BY_TYPE(backward_t, a.f.dtype, a.f.d, a, st);
}

}  // namespace gdr
