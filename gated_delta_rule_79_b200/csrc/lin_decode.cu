// One-token step of linear attention with one decay per head (sm_100a).
//
// Row r of the state S (d_v x d_k, fp32) of a (sequence, head) becomes
//
//     S[r,:] = a S[r,:] + v_r k,      o_r = S[r,:] . q
//
// Bound by HBM like the delta rule's step (decode.cu): the state is read and written once,
// 8 d_v d_k bytes against 5 flops an element.  The layout is the same too: a row is spread
// over 8 lanes, so a warp instruction moves four whole rows in 128-bit pieces and a dot
// product takes three shuffles.
//
// A warp updates d_v >> rshift rows.  rshift grows until the launch has about 16 warps for
// each SM (no part below 8 rows): the batch of 256 x 32 states runs with 1 (two warps a
// state), a single sequence of 32 heads with 4, which spreads its 2 MB over 128 CTAs.

#include "common.cuh"
#include "launch.h"

namespace gdr {
namespace {

constexpr int kWarps = 4;

template <int DK, typename T>
__global__ void __launch_bounds__(kWarps * 32)
lin_decode_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                  const float* __restrict__ decay, float* __restrict__ state,
                  T* __restrict__ o, int NH, int H, int dv, int rshift) {
  constexpr int LPR = 8;               // lanes per state row
  constexpr int RPW = 32 / LPR;        // rows per warp instruction
  constexpr int F4 = DK / (4 * LPR);   // float4 pieces per lane per row
  constexpr int ITER = 2;              // row groups in flight per warp

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long task = (long)blockIdx.x * kWarps + warp;
  if (task >= ((long)NH << rshift)) return;
  const long head = task >> rshift;
  const int part = (int)(task & ((1 << rshift) - 1));
  const int rows = dv >> rshift;
  const int sub = lane / LPR, j = lane % LPR;

  const long first = head * dv + (long)part * rows;
  float* Sh = state + first * DK;
  const T* vh = v + first;
  T* oh = o + first;
  const float a = decay[head % H];
  // this lane owns channels 4p..4p+3 for p = j + LPR*m, m < F4
  float4 kr[F4], qr[F4];
#pragma unroll
  for (int m = 0; m < F4; ++m) {
    const int c = 4 * (j + LPR * m);
    kr[m] = Elem<T>::load4(k + head * DK + c);
    qr[m] = Elem<T>::load4(q + head * DK + c);
  }
  for (int r0 = 0; r0 < rows; r0 += RPW * ITER) {
    float4 s[ITER][F4];
    float vr[ITER];
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const int row = r0 + it * RPW + sub;
#pragma unroll
      for (int m = 0; m < F4; ++m)
        s[it][m] = __ldcs(reinterpret_cast<const float4*>(Sh + (long)row * DK +
                                                          4 * (j + LPR * m)));
      vr[it] = Elem<T>::load(vh + row);
    }
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
      const int row = r0 + it * RPW + sub;
      float acc = 0.f;
#pragma unroll
      for (int m = 0; m < F4; ++m) {
        float4& x = s[it][m];
        x.x = fmaf(vr[it], kr[m].x, a * x.x);
        x.y = fmaf(vr[it], kr[m].y, a * x.y);
        x.z = fmaf(vr[it], kr[m].z, a * x.z);
        x.w = fmaf(vr[it], kr[m].w, a * x.w);
        acc = fmaf(x.x, qr[m].x, fmaf(x.y, qr[m].y, fmaf(x.z, qr[m].z, fmaf(x.w, qr[m].w, acc))));
        __stcs(reinterpret_cast<float4*>(Sh + (long)row * DK + 4 * (j + LPR * m)), x);
      }
#pragma unroll
      for (int off = 1; off < LPR; off <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
      if (j == 0) Elem<T>::store(oh + row, acc);
    }
  }
}

template <int DK, typename T>
cudaError_t launch_t(const LinDecodeArgs& a, cudaStream_t st) {
  const long NH = (long)a.N * a.H;
  int rshift = 1;
  while ((NH << rshift) < 148 * 16 && (a.dv >> (rshift + 1)) >= 8) ++rshift;
  const long tasks = NH << rshift;
  lin_decode_kernel<DK, T><<<(unsigned)((tasks + kWarps - 1) / kWarps), kWarps * 32, 0, st>>>(
      (const T*)a.q, (const T*)a.k, (const T*)a.v, a.decay, a.state, (T*)a.o, (int)NH, a.H, a.dv,
      rshift);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_dk(const LinDecodeArgs& a, cudaStream_t st) {
  switch (a.dk) {
    case 32: return launch_t<32, T>(a, st);
    case 64: return launch_t<64, T>(a, st);
    case 128: return launch_t<128, T>(a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_lin_decode(const LinDecodeArgs& a, cudaStream_t st) {
  return a.dtype == GDR_F32 ? launch_dk<float>(a, st) : launch_dk<__nv_bfloat16>(a, st);
}

}  // namespace gdr
