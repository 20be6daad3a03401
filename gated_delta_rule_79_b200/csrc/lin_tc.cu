// Linear attention with one decay per head on the tensor cores (sm_100a, tcgen05 + TMA): bf16
// tensors, d_k and d_v of 64 or 128.  The algebra, the scans and the two passes over the
// segments are in lin_common.cuh.
//
// Chunks of 64 tokens.  Everything that meets the state runs transposed, value rows in the 128
// TMEM lanes (d_v = 64 uses its one panel twice and ignores the upper lanes); a thread of warps
// 0-3 holds a row of the fp32 state in registers:
//
//     G  = Q K^T                        (64 x 64, bf16 operands as they are: exact products)
//     P  = G (.) a^(i_t - i_j), lower   (bf16)
//     O1 = S Q^T,  O2 = V^T P^T,        o = a^(i+E) O1 + O2
//     KV = V^T K~,                      K~ = a^(L-1-i) k
//     S  = a^(L-1+E) S + KV
//
// A bf16 product with decayed keys would carry a rounding of 2^-9 into the fp32 state, so K~
// enters as a sum of three bf16 terms (24 bits) whose products are exact, the smallest first.
// KV is a new accumulator for every chunk, added to S by an fp32 fma: the tensor cores truncate
// what they accumulate, and a state kept there lost 2e-7 of itself with each chunk of its memory
// (measured: 7e-6 after 4096 tokens at a decay of 1 - 2^-11).  S is rounded to bf16 for O1, P
// for O2: one rounding of an operand each, as the output's own.
//
// Bound: HBM, 2 (d_k + d_v) 2 bytes a token and head: 64 KB a chunk at d = 128, about 2800 cycles
// of an SM's share of 6.5 TB/s, against 1400 cycles of products (KV 768 of them) and passes of
// 200 to 600 cycles that run beside each other: warps 0-3 the state, 4-7 K~, 8-11 P and the
// outputs, 12 issues, 13 loads up to three chunks ahead.
//
// Waits are bounded: a give-up sets the status word, drains what is in flight and ends the CTA.

#include "attn_tc.cuh"
#include "lin_common.cuh"
#include "tma_host.h"

namespace gdr {
namespace {

using namespace attn;     // operand descriptors, bounded waits
using namespace lin;

constexpr int kC = 64;

__device__ __forceinline__ uint64_t* mb(unsigned long long& x) {
  return reinterpret_cast<uint64_t*>(&x);
}
__host__ __device__ constexpr uint32_t idesc_a_mn(uint32_t id) { return id | (1u << 15); }

// V^T as an A operand with M = 128: with one panel of 64 value rows both halves read it.
template <int DV>
__device__ __forceinline__ uint64_t v_as_a(uint32_t tile, int ks) {
  return sdesc(tile + (uint32_t)ks * 2048, DV == 128 ? kC * 128 : 0, 1024);
}

// One thread's share (pieces of eight channels) of K~ = weight(row) k as three bf16 tiles.
template <int DK, int THREADS, typename W>
__device__ __forceinline__ void split_keys(const unsigned char* k, unsigned char* kt, int t,
                                           W weight) {
  constexpr int TILE = kC * DK * 2;
#pragma unroll 2
  for (int e = t; e < kC * (DK / 8); e += THREADS) {
    // pieces of a panel row follow each other as stored: the swizzle only permutes them
    const int r = (e >> 3) % kC, pn = e / (8 * kC), at = pn * kC * 128 + r * 128 + (e & 7) * 16;
    const uint4 x = *reinterpret_cast<const uint4*>(k + at);
    const uint32_t* xs = reinterpret_cast<const uint32_t*>(&x);
    const float w = weight(r);
    uint4 out[3];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float u = __uint_as_float(xs[c] << 16) * w, v = __uint_as_float(xs[c] & 0xffff0000u) * w;
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(u, v);
        const uint32_t b = *reinterpret_cast<const uint32_t*>(&p);
        reinterpret_cast<uint32_t*>(&out[s])[c] = b;
        u -= __uint_as_float(b << 16);
        v -= __uint_as_float(b & 0xffff0000u);
      }
    }
    *reinterpret_cast<uint4*>(kt + at) = out[0];
    *reinterpret_cast<uint4*>(kt + TILE + at) = out[1];
    *reinterpret_cast<uint4*>(kt + 2 * TILE + at) = out[2];
  }
}

// ---- first pass: what a segment leaves in the state ---------------------------------------

template <int DK, int DV>
struct SegLayout {
  static constexpr int KT = kC * DK * 2, VT = kC * DV * 2;
  static constexpr int STAGE = KT + VT, STAGES = 3;
  static constexpr int SPLIT = STAGES * STAGE;           // K~, two of them
  static constexpr int PW = SPLIT + 2 * 3 * KT;          // a^n, n = 0 .. 63
  static constexpr int SMALL = PW + 256;
  static constexpr int SMEM = SMALL + 256 + 1024;
  static_assert(SMEM <= 232448, "shared memory");
};
struct SegSmall {
  unsigned long long full[3], empty[3], kt_full[2], kv_done[2], kv_free[2], drained;
  float far[3];                     // of each stage: a^(tokens of the segment after its chunk)
  uint32_t tmem;
  int abort;
};
constexpr int kLinWarps = 16;       // four warpgroups for the register split, 14 warps at work

struct LinMaps {
  CUtensorMap q[kLinMaxJobs], k[kLinMaxJobs], v[kLinMaxJobs];
};

template <int DK, int DV>
__global__ void __launch_bounds__(kLinWarps * 32, 1)
lin_segment_tc(const __grid_constant__ LinMaps maps, const LinScan sc, uint32_t spin) {
  using L = SegLayout<DK, DV>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  SegSmall& ss = *reinterpret_cast<SegSmall*>(sm + L::SMALL);
  float* pw = reinterpret_cast<float*>(sm + L::PW);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int job = blockIdx.y;
  const int rev = sc.job[job].rev;
  const int p = blockIdx.x % (sc.nseg - 1), bh = blockIdx.x / (sc.nseg - 1);
  const int b = bh / sc.H, h = bh % sc.H;
  const Segment sg = segment(p, rev, sc.T, sc.seg_len, sc.nseg);
  const int nch = (sg.n + kC - 1) / kC;
  const double l2 = log2_decay(sc.decay[h]);
  if (tid == 0) {
    for (int s = 0; s < 3; ++s) {
      mbar_init(mb(ss.full[s]), 1);
      mbar_init(mb(ss.empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(mb(ss.kt_full[s]), 8);
      mbar_init(mb(ss.kv_done[s]), 1);
      mbar_init(mb(ss.kv_free[s]), 4);
    }
    mbar_init(mb(ss.drained), 1);
    ss.abort = 0;
    fence_mbar_init();
  }
  if (tid < kC) pw[tid] = (float)decay_pow(l2, tid);
  if (warp == 0) tmem_alloc(&ss.tmem, 256);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tb = ss.tmem;
  const uint32_t sb = smem_u32(sm);
  const Waits wait{sc.status, &ss.abort, spin};

  // (a sum: the order of the chunks does not matter, they run as they lie)
  if (warp < 4) {
    more_registers<208>();
    // ---- the sum over the chunks: thread = value row ----------------------------------------
    const int v = warp * 32 + lane;
    const uint32_t tl = (uint32_t)(warp * 32) << 16;
    float S[DK];
#pragma unroll
    for (int e = 0; e < DK; ++e) S[e] = 0.f;
    bool ok = true;
    for (int c = 0; c < nch; ++c) {
      const int w = c & 1;
      if (!(ok = wait(mb(ss.kv_done[w]), (uint32_t)(c >> 1) & 1u))) break;
      fence_after_sync();
#pragma unroll
      for (int q = 0; q < DK / 32; ++q) {
        float x[32];
        tmem_ld32(tb + tl + 128 * w + 32 * q, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) S[32 * q + e] += x[e];
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb(ss.kv_free[w]));
    }
    if (ok && v < DV) {
      float* dst = sc.part + (((size_t)job * sc.B * sc.H + bh) * (sc.nseg - 1) + p) * DV * DK +
                   (size_t)v * DK;
#pragma unroll
      for (int e = 0; e < DK / 4; ++e)
        reinterpret_cast<float4*>(dst)[e] =
            make_float4(S[4 * e], S[4 * e + 1], S[4 * e + 2], S[4 * e + 3]);
    }
  } else if (warp < 12) {
    fewer_registers<112>();
    // ---- K~ ----------------------------------------------------------------------------------
    for (int c = 0; c < nch; ++c) {
      const int s = c % 3, w = c & 1;
      if (!wait(mb(ss.full[s]), (uint32_t)(c / 3) & 1u)) break;
      // the product of chunk c - 2 has read this buffer
      if (c >= 2 && !wait(mb(ss.kv_done[w]), (uint32_t)((c - 2) >> 1) & 1u)) break;
      const float far = ss.far[s];
      const int last = min(kC, sg.n - c * kC) - 1;
      split_keys<DK, 256>(sm + s * L::STAGE, sm + L::SPLIT + w * 3 * L::KT, tid - 128,
                          [&](int r) { return far * pw[rev ? r : max(last - r, 0)]; });
      fence_smem_to_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb(ss.kt_full[w]));
    }
  } else {
    fewer_registers<72>();
    if (warp == 12) {
      constexpr uint32_t id = idesc_a_mn(idesc_bf16_mn(128, DK));
      for (int c = 0; c < nch; ++c) {
        const int s = c % 3, w = c & 1;
        if (!wait(mb(ss.full[s]), (uint32_t)(c / 3) & 1u)) break;
        if (!wait(mb(ss.kt_full[w]), (uint32_t)(c >> 1) & 1u)) break;
        if (c >= 2 && !wait(mb(ss.kv_free[w]), (uint32_t)((c - 2) >> 1) & 1u)) break;
        fence_after_sync();
#pragma unroll
        for (int t = 2; t >= 0; --t)
#pragma unroll
          for (int ks = 0; ks < kC / 16; ++ks)
            mma_bf16_w(tb + 128 * w, v_as_a<DV>(sb + s * L::STAGE + L::KT, ks),
                       mnmajor(sb + L::SPLIT + (3 * w + t) * L::KT, kC, ks), id, t < 2 || ks > 0);
        mma_commit_w(mb(ss.kv_done[w]));
        mma_commit_w(mb(ss.empty[s]));
      }
      // the products issued here complete before tensor memory is freed
      mma_commit_w(mb(ss.drained));
      mbar_wait(mb(ss.drained), 0, kDrain);
    } else if (warp == 13) {
      int done = 0;
      for (int c = 0; c < nch; ++c) {
        const int s = c % 3;
        if (!wait(mb(ss.empty[s]), ((uint32_t)(c / 3) & 1u) ^ 1u)) break;
        const int t0 = sg.a + c * kC;
        if (lane == 0) {
          const int Lc = min(kC, sg.n - c * kC);
          const long after = rev ? c * kC : sg.n - c * kC - Lc;
          ss.far[s] = (float)decay_pow(l2, after);
          mbar_expect_tx(mb(ss.full[s]), L::STAGE);
          for (int pn = 0; pn < DK / 64; ++pn)
            tma_load_4d(sb + s * L::STAGE + pn * kC * 128, &maps.k[job], 64 * pn, h, t0, b,
                        mb(ss.full[s]));
          for (int pn = 0; pn < DV / 64; ++pn)
            tma_load_4d(sb + s * L::STAGE + L::KT + pn * kC * 128, &maps.v[job], 64 * pn, h, t0,
                        b, mb(ss.full[s]));
        }
        done = c + 1;
      }
      // copies in flight land before the CTA leaves, also when some warp gave up
      if (lane == 0)
        for (int c = max(0, done - 3); c < done; ++c)
          mbar_wait(mb(ss.full[c % 3]), (uint32_t)(c / 3) & 1u, kDrain);
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tb, 256);
}

// ---- second pass: the outputs -----------------------------------------------------------------

template <int DK, int DV>
struct OutLayout {
  static constexpr int KT = kC * DK * 2, VT = kC * DV * 2;
  static constexpr int STAGE = 2 * KT + VT, STAGES = 3;  // q, k, v
  static constexpr int SPLIT = STAGES * STAGE;
  static constexpr int P = SPLIT + 3 * KT;               // bf16 [64 t][64 j], two of them
  static constexpr int PW = P + 2 * 8192;                // a^n, n = 0 .. 64
  static constexpr int SMALL = PW + 512;
  static constexpr int SMEM = SMALL + 512 + 1024;
  static_assert(SMEM <= 232448, "shared memory");
  // tensor memory
  static constexpr uint32_t KV = 0;                      // DK columns
  static constexpr uint32_t SB = 128;                    // the state in bf16, DK / 2 columns
  static constexpr uint32_t G = 192;
  static constexpr uint32_t O1 = 256, O2 = 384;          // + 64 * (chunk & 1)
};
struct OutSmall {
  unsigned long long full[3], empty[3];
  unsigned long long g_full, p_full[2], kt_full, kv_done, kv_free, s_ready, o1_done, o_full[2],
      o_free[2], drained;
  uint32_t tmem;
  int abort;
};

template <int DK, int DV>
__global__ void __launch_bounds__(kLinWarps * 32, 1)
lin_out_tc(const __grid_constant__ LinMaps maps, const LinScan sc, uint32_t spin) {
  using L = OutLayout<DK, DV>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  OutSmall& os = *reinterpret_cast<OutSmall*>(sm + L::SMALL);
  float* pw = reinterpret_cast<float*>(sm + L::PW);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int job = blockIdx.y;
  const int rev = sc.job[job].rev, e0 = sc.job[job].e0;
  const int p = blockIdx.x % sc.nseg, bh = blockIdx.x / sc.nseg;
  const int b = bh / sc.H, h = bh % sc.H;
  const Segment sg = segment(p, rev, sc.T, sc.seg_len, sc.nseg);
  const int nch = (sg.n + kC - 1) / kC;
  const double l2 = log2_decay(sc.decay[h]);
  float* s_out = p == sc.nseg - 1 ? sc.job[job].s_out : nullptr;
  const int nstate = s_out ? nch : nch - 1;        // chunks whose KV is needed
  if (tid == 0) {
    for (int s = 0; s < 3; ++s) {
      mbar_init(mb(os.full[s]), 1);
      mbar_init(mb(os.empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(mb(os.p_full[s]), 4);
      mbar_init(mb(os.o_full[s]), 1);
      mbar_init(mb(os.o_free[s]), 4);
    }
    mbar_init(mb(os.g_full), 1);
    mbar_init(mb(os.kt_full), 4);
    mbar_init(mb(os.s_ready), 4);
    mbar_init(mb(os.kv_done), 1);
    mbar_init(mb(os.kv_free), 4);
    mbar_init(mb(os.o1_done), 1);
    mbar_init(mb(os.drained), 1);
    os.abort = 0;
    fence_mbar_init();
  }
  if (tid <= kC) pw[tid] = (float)decay_pow(l2, tid);
  if (warp == 0) tmem_alloc(&os.tmem, 512);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tb = os.tmem;
  const uint32_t sb = smem_u32(sm);
  const Waits wait{sc.status, &os.abort, spin};
  // chunk c in processing order: its first token in the segment
  auto chunk_at = [&](int c) { return (rev ? nch - 1 - c : c) * kC; };

  if (warp < 4) {
    more_registers<208>();
    // ---- the state: thread = value row ----------------------------------------------------
    const int v = warp * 32 + lane;
    const uint32_t tl = (uint32_t)(warp * 32) << 16;
    // entering: the call's own state decayed over the tokens before, and what the earlier
    // segments left
    float S[DK];
#pragma unroll
    for (int e = 0; e < DK; ++e) S[e] = 0.f;
    if (v < DV) {
      const LinJob& jb = sc.job[job];
      if (jb.s_in) {
        const float f = p == 0 ? 1.f : (float)decay_pow(l2, (long)sg.before + e0 - 1);
        const float* s = jb.s_in + (size_t)bh * DV * DK;
        if (jb.s_trans) {
#pragma unroll
          for (int e = 0; e < DK; ++e) S[e] = f * s[(size_t)e * DV + v];
        } else {
#pragma unroll
          for (int e = 0; e < DK / 4; ++e) {
            const float4 y = *reinterpret_cast<const float4*>(s + (size_t)v * DK + 4 * e);
            S[4 * e] = f * y.x;
            S[4 * e + 1] = f * y.y;
            S[4 * e + 2] = f * y.z;
            S[4 * e + 3] = f * y.w;
          }
        }
      }
      const float* part = sc.part +
                          ((size_t)job * sc.B * sc.H + bh) * (sc.nseg - 1) * DV * DK +
                          (size_t)v * DK;
      for (int m = 0; m < p; ++m) {
        const Segment pm = segment(m, rev, sc.T, sc.seg_len, sc.nseg);
        const float f = (float)decay_pow(l2, (long)sg.before - pm.before - pm.n);
        const float* s = part + (size_t)m * DV * DK;
#pragma unroll
        for (int e = 0; e < DK / 4; ++e) {
          const float4 y = *reinterpret_cast<const float4*>(s + 4 * e);
          S[4 * e] = fmaf(f, y.x, S[4 * e]);
          S[4 * e + 1] = fmaf(f, y.y, S[4 * e + 1]);
          S[4 * e + 2] = fmaf(f, y.z, S[4 * e + 2]);
          S[4 * e + 3] = fmaf(f, y.w, S[4 * e + 3]);
        }
      }
    }
    bool ok = true;
    for (int c = 0; c < nch; ++c) {
      // the bf16 copy, once O1 of the chunk before has read the last one
      if (c > 0 && !(ok = wait(mb(os.o1_done), (uint32_t)(c - 1) & 1u))) break;
      fence_after_sync();
#pragma unroll
      for (int q = 0; q < DK / 64; ++q) {
        float y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = pack2(S[64 * q + 2 * e], S[64 * q + 2 * e + 1]);
        tmem_st32(tb + tl + L::SB + 32 * q, y);
      }
      tmem_wait_st();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb(os.s_ready));
      if (c >= nstate) break;
      const int E = p == 0 && c == 0 ? e0 : 1;
      const int Lc = min(kC, sg.n - chunk_at(c));
      // the chunk's decay as a pair of floats: its rounding would otherwise be the same in
      // every chunk and add up over a long prompt
      const double fd = decay_pow(l2, (long)Lc - 1 + E);
      const float fh = (float)fd, fl = (float)(fd - (double)fh);
      if (!(ok = wait(mb(os.kv_done), (uint32_t)c & 1u))) break;
      fence_after_sync();
#pragma unroll
      for (int q = 0; q < DK / 32; ++q) {
        float x[32];
        tmem_ld32(tb + tl + L::KV + 32 * q, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e)
          S[32 * q + e] = fmaf(fh, S[32 * q + e], fmaf(fl, S[32 * q + e], x[e]));
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb(os.kv_free));
    }
    if (s_out && ok && v < DV) {
      const float f = (float)decay_pow(l2, 1 - e0);
      float* dst = s_out + (size_t)bh * DV * DK + (size_t)v * DK;
#pragma unroll
      for (int e = 0; e < DK / 4; ++e)
        reinterpret_cast<float4*>(dst)[e] = make_float4(f * S[4 * e], f * S[4 * e + 1],
                                                        f * S[4 * e + 2], f * S[4 * e + 3]);
    }
  } else if (warp < 8) {
    fewer_registers<112>();
    // ---- K~ ----------------------------------------------------------------------------------
    for (int c = 0; c < nstate; ++c) {
      const int s = c % 3;
      if (!wait(mb(os.full[s]), (uint32_t)(c / 3) & 1u)) break;
      if (c > 0 && !wait(mb(os.kv_done), (uint32_t)(c - 1) & 1u)) break;
      const int last = min(kC, sg.n - chunk_at(c)) - 1;
      split_keys<DK, 128>(sm + s * L::STAGE + L::KT, sm + L::SPLIT, tid - 128,
                          [&](int r) { return pw[rev ? r : max(last - r, 0)]; });
      fence_smem_to_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb(os.kt_full));
    }
  } else if (warp < 12) {
    fewer_registers<112>();
    // ---- P of chunk c, then the outputs of chunk c - 1 ----------------------------------------
    const int q4 = warp & 3;
    const uint32_t tl = (uint32_t)(q4 * 32) << 16;
    const int v = q4 * 32 + lane;
    __nv_bfloat16* ob =
        (__nv_bfloat16*)sc.job[job].o + (((size_t)b * sc.T + sg.a) * sc.H + h) * DV;
    for (int c = 0; c <= nch; ++c) {
      if (c < nch) {
        if (!wait(mb(os.g_full), (uint32_t)c & 1u)) break;
        fence_after_sync();
        // an M = 64 accumulator: row t in lane 32 (t / 16) + t % 16.  P's buffer was last read
        // by the product of chunk c - 2, which came before this Gram
        const int t = 16 * q4 + (lane & 15);
        unsigned char* pt = sm + L::P + (c & 1) * 8192 + t * 128;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x[32];
          tmem_ld32(tb + tl + L::G + 32 * half, x);
          tmem_wait_ld();
          if (lane < 16) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int gap = rev ? 32 * half + e - t : t - (32 * half + e);
              x[e] = gap >= 0 ? x[e] * pw[gap] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<float4*>(pt + (((4 * half + e) ^ (t & 7)) << 4)) =
                  make_float4(pack2(x[8 * e], x[8 * e + 1]), pack2(x[8 * e + 2], x[8 * e + 3]),
                              pack2(x[8 * e + 4], x[8 * e + 5]),
                              pack2(x[8 * e + 6], x[8 * e + 7]));
          }
        }
        fence_smem_to_async();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(mb(os.p_full[c & 1]));
      }
      if (c > 0) {
        const int d = c - 1, w = d & 1;
        if (!wait(mb(os.o_full[w]), (uint32_t)(d >> 1) & 1u)) break;
        fence_after_sync();
        const int x0 = chunk_at(d), Lc = min(kC, sg.n - x0);
        const int E = p == 0 && d == 0 ? e0 : 1;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x[32], y[32];
          tmem_ld32(tb + tl + L::O1 + 64 * w + 32 * half, x);
          tmem_ld32(tb + tl + L::O2 + 64 * w + 32 * half, y);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int r = 32 * half + e;
            x[e] = fmaf(x[e], pw[rev ? max(Lc - 1 - r, 0) + E : r + E], y[e]);
          }
          // two lanes swap halves, so that each stores two neighbouring channels of one token
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const bool odd = lane & 1;
            const float got = __shfl_xor_sync(0xffffffffu, odd ? x[e] : x[e + 1], 1);
            const float two = odd ? pack2(got, x[e + 1]) : pack2(x[e], got);
            const int r = 32 * half + e + odd;
            if (r < Lc && v < DV)
              *reinterpret_cast<float*>(ob + (size_t)(x0 + r) * sc.H * DV + (v & ~1)) = two;
          }
        }
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(mb(os.o_free[w]));
      }
    }
  } else {
    fewer_registers<72>();
    if (warp == 12) {
      // ---- issuing warp --------------------------------------------------------------------------
      constexpr uint32_t id_g = idesc_bf16(64, 64), id_o1 = idesc_bf16(128, 64),
                         id_o2 = idesc_a_mn(idesc_bf16(128, 64)),
                         id_kv = idesc_a_mn(idesc_bf16_mn(128, DK));
      for (int c = 0; c <= nch; ++c) {
        const int s = c % 3, w = c & 1;
        const uint32_t at = sb + s * L::STAGE;
        if (c < nch) {
          if (!wait(mb(os.full[s]), (uint32_t)(c / 3) & 1u)) break;
          // G is free once P of the chunk before has been formed
          if (c > 0 && !wait(mb(os.p_full[w ^ 1]), (uint32_t)((c - 1) >> 1) & 1u)) break;
          fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            mma_bf16_w(tb + L::G, kmajor(at, kC, ks), kmajor(at + L::KT, kC, ks), id_g, ks > 0);
          mma_commit_w(mb(os.g_full));
        }
        if (c > 0) {
          // O2 of chunk c - 1
          const int d = c - 1, sd = d % 3, wd = d & 1;
          if (c == nch && !wait(mb(os.p_full[wd]), (uint32_t)(d >> 1) & 1u)) break;
          fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < kC / 16; ++ks)
            mma_bf16_w(tb + L::O2 + 64 * wd, v_as_a<DV>(sb + sd * L::STAGE + 2 * L::KT, ks),
                       kmajor(sb + L::P + wd * 8192, kC, ks), id_o2, ks > 0);
          mma_commit_w(mb(os.o_full[wd]));
          mma_commit_w(mb(os.empty[sd]));
        }
        if (c < nstate) {
          // the accumulator is free once the state has taken the chunk before
          if (!wait(mb(os.kt_full), (uint32_t)c & 1u)) break;
          if (c > 0 && !wait(mb(os.kv_free), (uint32_t)(c - 1) & 1u)) break;
          fence_after_sync();
#pragma unroll
          for (int t = 2; t >= 0; --t)
#pragma unroll
            for (int ks = 0; ks < kC / 16; ++ks)
              mma_bf16_w(tb + L::KV, v_as_a<DV>(at + 2 * L::KT, ks),
                         mnmajor(sb + L::SPLIT + t * L::KT, kC, ks), id_kv, t < 2 || ks > 0);
          mma_commit_w(mb(os.kv_done));
        }
        if (c < nch) {
          if (!wait(mb(os.s_ready), (uint32_t)c & 1u)) break;
          if (c >= 2 && !wait(mb(os.o_free[w]), (uint32_t)((c - 2) >> 1) & 1u)) break;
          fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            mma_bf16_ta_w(tb + L::O1 + 64 * w, tb + L::SB + 8 * ks, kmajor(at, kC, ks), id_o1,
                          ks > 0);
          mma_commit_w(mb(os.o1_done));
        }
      }
      // the products issued here complete before tensor memory is freed
      mma_commit_w(mb(os.drained));
      mbar_wait(mb(os.drained), 0, kDrain);
    } else if (warp == 13) {
      // ---- loader -----------------------------------------------------------------------------------
      int done = 0;
      for (int c = 0; c < nch; ++c) {
        const int s = c % 3;
        if (!wait(mb(os.empty[s]), ((uint32_t)(c / 3) & 1u) ^ 1u)) break;
        if (lane == 0) {
          const uint32_t at = sb + s * L::STAGE;
          const int t0 = sg.a + chunk_at(c);
          uint64_t* bar = mb(os.full[s]);
          mbar_expect_tx(bar, L::STAGE);
          for (int pn = 0; pn < DK / 64; ++pn) {
            tma_load_4d(at + pn * kC * 128, &maps.q[job], 64 * pn, h, t0, b, bar);
            tma_load_4d(at + L::KT + pn * kC * 128, &maps.k[job], 64 * pn, h, t0, b, bar);
          }
          for (int pn = 0; pn < DV / 64; ++pn)
            tma_load_4d(at + 2 * L::KT + pn * kC * 128, &maps.v[job], 64 * pn, h, t0, b, bar);
        }
        done = c + 1;
      }
      // copies in flight land before the CTA leaves, also when some warp gave up
      if (lane == 0)
        for (int c = max(0, done - 3); c < done; ++c)
          mbar_wait(mb(os.full[c % 3]), (uint32_t)(c / 3) & 1u, kDrain);
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tb, 512);
}

template <int DK, int DV>
cudaError_t launch_t(const LinScan& sc, cudaStream_t st) {
  LinMaps maps;
  for (int j = 0; j < sc.njobs; ++j)
    if (!encode_bthd_bf16(&maps.q[j], sc.job[j].q, sc.B, sc.T, sc.H, DK, 64, kC, true) ||
        !encode_bthd_bf16(&maps.k[j], sc.job[j].k, sc.B, sc.T, sc.H, DK, 64, kC, true) ||
        !encode_bthd_bf16(&maps.v[j], sc.job[j].v, sc.B, sc.T, sc.H, DV, 64, kC, true))
      return cudaErrorInvalidValue;
  const uint32_t spin = attn_spin_limit();
  cudaError_t e;
  if (sc.nseg > 1) {
    auto kern = lin_segment_tc<DK, DV>;
    constexpr int smem = SegLayout<DK, DV>::SMEM;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<dim3((unsigned)(sc.B * sc.H * (sc.nseg - 1)), sc.njobs), kLinWarps * 32, smem, st>>>(
        maps, sc, spin);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  auto kern = lin_out_tc<DK, DV>;
  constexpr int smem = OutLayout<DK, DV>::SMEM;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<dim3((unsigned)(sc.B * sc.H * sc.nseg), sc.njobs), kLinWarps * 32, smem, st>>>(maps, sc,
                                                                                       spin);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_tc(const LinScan& sc, cudaStream_t st) {
  if (sc.dk == 128) return sc.dv == 128 ? launch_t<128, 128>(sc, st) : launch_t<128, 64>(sc, st);
  return sc.dv == 128 ? launch_t<64, 128>(sc, st) : launch_t<64, 64>(sc, st);
}

}  // namespace gdr
