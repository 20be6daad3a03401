// Linear attention with one decay per head on the CUDA cores, all in fp32: fp32 tensors,
// and head sizes the tensor-core kernels do not take (lin_tc.cu).  The algebra and the two
// passes over the segments are in lin_common.cuh.
//
// Chunks of 32 tokens.  A thread of the 16 x 16 grid keeps (d_v / 16) x (d_k / 16) elements
// of the state in registers; the outputs' kernel mirrors the state in shared memory for S q.
// Bound: fp32 multiply-adds, 2 (2 d_k d_v + 16 (d_k + d_v)) flops a token, with the reads of the
// operands from shared memory close behind: four neighbours to a read, the threads of a warp as
// 4 x 8 where a product reads both operands there.  A CTA of d = 128 has an SM to itself, so its
// loads do not hide behind another's work: they run a chunk ahead.  Multiply-adds go two to
// an instruction, over neighbouring columns or over even and odd channels.  2 x 2048 tokens, 8
// heads of 128 x 128, fp32: 154 us; one multiply-add an instruction 167, with loads that the chunk
// waits for 216, with 2 x 16 threads 232 as well (6 heads of 64 x 128, gradients: 144 and 152).  With
// 32 x 32 the state's sums are short chains that pairs make longer: gradients of 4 x 4096 tokens, 16
// heads, take 503 us against 525 with one multiply-add an instruction, but those of 2 x 1000 tokens,
// 4 heads, which fill no SM, 31.2 against 28.7 (a prompt of either: 200 and 209, 22 and 22).

#include "attn_common.cuh"
#include "lin_common.cuh"
#include "once.h"

namespace gdr {
namespace {

using namespace lin;
using attn::fma2;
using attn::mul2;

constexpr int kC = 32;
constexpr int kThreads = 256;

// N = D / 16 elements a thread of D: column j of thread tx, four (or two) neighbours at a time,
// and row i of thread ty, N neighbours.
template <int D>
struct Share {
  static constexpr int N = D / 16, W = N < 4 ? N : 4;
  static __device__ __forceinline__ int col(int tx, int j) {
    return tx * W + 16 * W * (j / W) + j % W;
  }
  // the W neighbours from column col(tx, j) on
  static __device__ __forceinline__ void put(float* p, const float* x) {
    if constexpr (W == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
  }
  static __device__ __forceinline__ void cols(const float* r, int tx, float (&x)[N]) {
#pragma unroll
    for (int j = 0; j < N; j += W) read(r + col(tx, j), &x[j]);
  }
  static __device__ __forceinline__ void rows(const float* r, int ty, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += W) read(r + ty * N + i, &x[i]);
  }

 private:
  static __device__ __forceinline__ void read(const float* p, float* x) {
    if constexpr (W == 4) {
      const float4 f = *reinterpret_cast<const float4*>(p);
      x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
    } else {
      const float2 f = *reinterpret_cast<const float2*>(p);
      x[0] = f.x, x[1] = f.y;
    }
  }
};

// A chunk's rows of one operand on their way from global to shared memory, in registers while
// the chunk before it is worked on.  Rows from `end` on are zero.
template <typename T, int D>
struct Ahead {
  static constexpr int N = kC * (D / 4) / kThreads;
  float4 x[N];
  __device__ __forceinline__ void load(const T* src, size_t stride, int r0, int end, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = tid + i * kThreads, r = r0 + e / (D / 4), c = e % (D / 4) * 4;
      x[i] = r < end ? Elem<T>::load4(src + (size_t)r * stride + c)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void put(float* dst, int tid) const {       // rows of D + 4
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = tid + i * kThreads;
      *reinterpret_cast<float4*>(dst + e / (D / 4) * (D + 4) + e % (D / 4) * 4) = x[i];
    }
  }
};

// S[i][j] += w v_i k_j for one token; S holds pairs of neighbouring columns
template <int DK, int DV>
__device__ __forceinline__ void add_token(float2 (&S)[DV / 16][DK / 32], const float* k,
                                          const float* v, float w, int ty, int tx) {
  float kk[DK / 16], vv[DV / 16];
  Share<DK>::cols(k, tx, kk);
  Share<DV>::rows(v, ty, vv);
  float2 k2[DK / 32];
#pragma unroll
  for (int j = 0; j < DK / 32; ++j)
    k2[j] = mul2(make_float2(kk[2 * j], kk[2 * j + 1]), make_float2(w, w));
#pragma unroll
  for (int i = 0; i < DV / 16; ++i)
#pragma unroll
    for (int j = 0; j < DK / 32; ++j) S[i][j] = fma2(make_float2(vv[i], vv[i]), k2[j], S[i][j]);
}

// The sum over the segment's tokens of a^(n-1-i) v_i k_i^T.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kThreads)
lin_segment_simt(const LinScan sc) {
  const LinJob& jb = sc.job[blockIdx.y];
  __shared__ float ks[kC][DK + 4], vs[kC][DV + 4], near[kC];
  const int p = blockIdx.x % (sc.nseg - 1), bh = blockIdx.x / (sc.nseg - 1);
  const int b = bh / sc.H, h = bh % sc.H;
  const Segment sg = segment(p, jb.rev, sc.T, sc.seg_len, sc.nseg);
  const double l2 = log2_decay(sc.decay[h]);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  let_next_start();
  if (tid < kC) near[tid] = (float)decay_pow(l2, tid);
  float2 acc[DV / 16][DK / 32] = {};
  const T* kb = (const T*)jb.k + (((size_t)b * sc.T + sg.a) * sc.H + h) * DK;
  const T* vb = (const T*)jb.v + (((size_t)b * sc.T + sg.a) * sc.H + h) * DV;
  Ahead<T, DK> ka;
  Ahead<T, DV> va;
  ka.load(kb, (size_t)sc.H * DK, 0, sg.n, tid);
  va.load(vb, (size_t)sc.H * DV, 0, sg.n, tid);
  for (int x0 = 0; x0 < sg.n; x0 += kC) {
    const int L = min(kC, sg.n - x0);
    const float far = (float)decay_pow(l2, jb.rev ? x0 : sg.n - x0 - L);
    __syncthreads();
    ka.put(ks[0], tid);
    va.put(vs[0], tid);
    __syncthreads();
    ka.load(kb, (size_t)sc.H * DK, x0 + kC, sg.n, tid);
    va.load(vb, (size_t)sc.H * DV, x0 + kC, sg.n, tid);
#pragma unroll 4
    for (int r = 0; r < kC; ++r)
      add_token<DK, DV>(acc, ks[r], vs[r], near[jb.rev ? r : max(L - 1 - r, 0)] * far, ty, tx);
  }
  float* dst = sc.part + (((size_t)blockIdx.y * sc.B * sc.H + bh) * sc.nseg + p + 1) * DV * DK;
#pragma unroll
  for (int i = 0; i < DV / 16; ++i)
#pragma unroll
    for (int j = 0; j < DK / 16; j += Share<DK>::W)
      Share<DK>::put(dst + (ty * (DV / 16) + i) * DK + Share<DK>::col(tx, j), &acc[i][j / 2].x);
}

template <int DK, int DV>
struct OutSmem {
  float st[DV][DK + 4];          // the state entering the chunk
  float q[kC][DK + 4], k[kC][DK + 4], v[kC][DV + 4];
  float p[kC][kC + 4];
  float pw[kC + 1];              // a^n, n = 0 .. 32
};

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kThreads)
lin_out_simt(const LinScan sc) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  OutSmem<DK, DV>& sm = *reinterpret_cast<OutSmem<DK, DV>*>(smem_raw);
  const LinJob& jb = sc.job[blockIdx.y];
  const int p = blockIdx.x % sc.nseg, bh = blockIdx.x / sc.nseg;
  const int b = bh / sc.H, h = bh % sc.H;
  const Segment sg = segment(p, jb.rev, sc.T, sc.seg_len, sc.nseg);
  const double l2 = log2_decay(sc.decay[h]);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  if (tid <= kC) sm.pw[tid] = (float)decay_pow(l2, tid);

  // state entering the segment: what lin_carry.cu left for it, or the call's own if it is the
  // only one
  wait_for_previous();
  float2 S[DV / 16][DK / 32] = {};
  const bool parts = sc.nseg > 1;
  if (parts || jb.s_in) {
    const float* s =
        parts ? sc.part + (((size_t)blockIdx.y * sc.B * sc.H + bh) * sc.nseg + p) * DV * DK
              : jb.s_in + (size_t)bh * DV * DK;
#pragma unroll
    for (int i = 0; i < DV / 16; ++i)
#pragma unroll
      for (int j = 0; j < DK / 32; ++j) {
        const int r = ty * (DV / 16) + i, c = Share<DK>::col(tx, 2 * j);
        const bool turned = !parts && jb.s_trans;
        S[i][j] = make_float2(s[turned ? c * DV + r : r * DK + c],
                              s[turned ? (c + 1) * DV + r : r * DK + c + 1]);
      }
  }

  const size_t row0 = ((size_t)b * sc.T + sg.a) * sc.H + h;
  const T* qb = (const T*)jb.q + row0 * DK;
  const T* kb = (const T*)jb.k + row0 * DK;
  const T* vb = (const T*)jb.v + row0 * DV;
  T* ob = (T*)jb.o + row0 * DV;
  const int nch = (sg.n + kC - 1) / kC;
  Ahead<T, DK> qa, ka;
  Ahead<T, DV> va;
  auto ahead = [&](int ci) {
    if (ci >= nch) return;             // (the chunk behind the last would start below row 0)
    const int x = (jb.rev ? nch - 1 - ci : ci) * kC;
    qa.load(qb, (size_t)sc.H * DK, x, sg.n, tid);
    ka.load(kb, (size_t)sc.H * DK, x, sg.n, tid);
    va.load(vb, (size_t)sc.H * DV, x, sg.n, tid);
  };
  ahead(0);
  for (int ci = 0; ci < nch; ++ci) {
    const int x0 = (jb.rev ? nch - 1 - ci : ci) * kC;
    const int L = min(kC, sg.n - x0);
    const int E = (p == 0 && ci == 0) ? jb.e0 : 1;
    __syncthreads();
    qa.put(sm.q[0], tid);
    ka.put(sm.k[0], tid);
    va.put(sm.v[0], tid);
#pragma unroll
    for (int i = 0; i < DV / 16; ++i)
#pragma unroll
      for (int j = 0; j < DK / 16; j += Share<DK>::W)
        Share<DK>::put(&sm.st[ty * (DV / 16) + i][Share<DK>::col(tx, j)], &S[i][j / 2].x);
    __syncthreads();
    ahead(ci + 1);
    {
      const int t = tid >> 3, j0 = tid & 7;
      float2 g[4] = {};          // even and odd channels
#pragma unroll 4
      for (int c = 0; c < DK; c += 4) {
        const float4 a = *reinterpret_cast<const float4*>(&sm.q[t][c]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float4 d = *reinterpret_cast<const float4*>(&sm.k[j0 + 8 * m][c]);
          g[m] = fma2(make_float2(a.x, a.y), make_float2(d.x, d.y), g[m]);
          g[m] = fma2(make_float2(a.z, a.w), make_float2(d.z, d.w), g[m]);
        }
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int gap = jb.rev ? j0 + 8 * m - t : t - (j0 + 8 * m);
        sm.p[t][j0 + 8 * m] = gap >= 0 ? (g[m].x + g[m].y) * sm.pw[gap] : 0.f;
      }
    }
    __syncthreads();
    {
      // four rows and DV / 32 columns a thread: rows lr + 4 a of a warp's 16, columns lc + 8 b
      // of its DV / 4, so that a read serves a warp from one line of banks
      constexpr int NB = DV / 32;
      const int warp = tid >> 5, lr = (tid >> 3) & 3, lc = tid & 7;
      const int t0 = 16 * (warp & 1) + lr, c0 = (warp >> 1) * (DV / 4) + lc;
      float o[4][NB];
      float2 o2[4][NB] = {};
#pragma unroll 4
      for (int c = 0; c < DK; c += 4) {
        float4 u[4], w[NB];
#pragma unroll
        for (int x = 0; x < 4; ++x) u[x] = *reinterpret_cast<const float4*>(&sm.q[t0 + 4 * x][c]);
#pragma unroll
        for (int x = 0; x < NB; ++x) w[x] = *reinterpret_cast<const float4*>(&sm.st[c0 + 8 * x][c]);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int y = 0; y < NB; ++y) {
            o2[x][y] = fma2(make_float2(u[x].x, u[x].y), make_float2(w[y].x, w[y].y), o2[x][y]);
            o2[x][y] = fma2(make_float2(u[x].z, u[x].w), make_float2(w[y].z, w[y].w), o2[x][y]);
          }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int t = t0 + 4 * x, i = jb.rev ? L - 1 - t : t;
        const float f = t < L ? sm.pw[i + E] : 0.f;
#pragma unroll
        for (int y = 0; y < NB; ++y) o[x][y] = f * (o2[x][y].x + o2[x][y].y);
      }
#pragma unroll 2
      for (int j = 0; j < kC; j += 4) {          // rows past L are zero
        float pp[4][4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          *reinterpret_cast<float4*>(pp[x]) = *reinterpret_cast<const float4*>(&sm.p[t0 + 4 * x][j]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int y = 0; y < NB; ++y) {
            const float v = sm.v[j + e][c0 + 8 * y];
#pragma unroll
            for (int x = 0; x < 4; ++x) o[x][y] = fmaf(pp[x][e], v, o[x][y]);
          }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (t0 + 4 * x < L) {
          T* dst = ob + (size_t)(x0 + t0 + 4 * x) * sc.H * DV + c0;
#pragma unroll
          for (int y = 0; y < NB; ++y) Elem<T>::store(dst + 8 * y, o[x][y]);
        }
    }
    // the chunk's decay as a pair of floats: its rounding would otherwise be the same in
    // every chunk and add up over a long prompt
    const double fd = decay_pow(l2, (long)L - 1 + E);
    const float fh = (float)fd, fl = (float)(fd - (double)fh);
#pragma unroll
    for (int i = 0; i < DV / 16; ++i)
#pragma unroll
      for (int j = 0; j < DK / 32; ++j)
        S[i][j] = fma2(make_float2(fh, fh), S[i][j], mul2(make_float2(fl, fl), S[i][j]));
#pragma unroll 4
    for (int r = 0; r < kC; ++r)            // rows past L are zero
      add_token<DK, DV>(S, sm.k[r], sm.v[r], sm.pw[jb.rev ? r : max(L - 1 - r, 0)], ty, tx);
  }
  if (jb.s_out && p == sc.nseg - 1) {
    const float f = (float)decay_pow(l2, 1 - jb.e0);
    float* s = jb.s_out + (size_t)bh * DV * DK;
#pragma unroll
    for (int i = 0; i < DV / 16; ++i)
#pragma unroll
      for (int j = 0; j < DK / 32; ++j) {
        float* at = s + (ty * (DV / 16) + i) * DK + Share<DK>::col(tx, 2 * j);
        at[0] = f * S[i][j].x;
        at[1] = f * S[i][j].y;
      }
  }
}

template <typename T, int DK, int DV>
cudaError_t launch_t(const LinScan& sc, cudaStream_t st) {
  if (sc.nseg > 1) {
    lin_segment_simt<T, DK, DV>
        <<<dim3((unsigned)(sc.B * sc.H * (sc.nseg - 1)), sc.njobs), kThreads, 0, st>>>(sc);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_lin_carry(sc, st);
    if (e != cudaSuccess) return e;
  }
  constexpr int smem = (int)sizeof(OutSmem<DK, DV>);
  auto kern = lin_out_simt<T, DK, DV>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(sc.B * sc.H * sc.nseg), sc.njobs);
  if (sc.nseg > 1) return launch_after(kern, grid, kThreads, smem, st, sc);
  kern<<<grid, kThreads, smem, st>>>(sc);
  return cudaGetLastError();
}

// (bf16 with both head sizes 64 or 128 runs on the tensor cores)
template <typename T, int DK>
cudaError_t launch_dv(const LinScan& sc, cudaStream_t st) {
  if (sc.dv == 32) return launch_t<T, DK, 32>(sc, st);
  if constexpr (sizeof(T) == 4 || DK == 32) {
    if (sc.dv == 64) return launch_t<T, DK, 64>(sc, st);
    if (sc.dv == 128) return launch_t<T, DK, 128>(sc, st);
  }
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_dk(const LinScan& sc, cudaStream_t st) {
  switch (sc.dk) {
    case 32: return launch_dv<T, 32>(sc, st);
    case 64: return launch_dv<T, 64>(sc, st);
    case 128: return launch_dv<T, 128>(sc, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_lin_simt(const LinScan& sc, cudaStream_t st) {
  return sc.dtype == GDR_F32 ? launch_dk<float>(sc, st) : launch_dk<__nv_bfloat16>(sc, st);
}

}  // namespace gdr
