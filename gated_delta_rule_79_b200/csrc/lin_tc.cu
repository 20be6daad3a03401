// Linear attention with one decay per head on the tensor cores (sm_100a, tcgen05 + TMA): bf16
// tensors, d_k and d_v of 64 or 128.  The algebra, the scans and the two passes over the
// segments are in lin_common.cuh.
//
// Chunks of 64 tokens.  Everything that meets the state runs transposed, value rows in the 128
// TMEM lanes (d_v = 64 uses its one panel twice and ignores the upper lanes); two threads hold a
// row of the fp32 state in registers:
//
//     G  = Q K^T                        (64 x 64, bf16 operands as they are: exact products)
//     P  = G (.) a^(i_t - i_j), lower   (bf16)
//     O1 = S Q^T,  O2 = V^T P^T,        o = a^(i+E) O1 + O2
//     KV = V~^T K,                      V~ = a^(L-1-i) v
//     S  = a^(L-1+E) S + KV
//
// A bf16 product with decayed values would carry a rounding of 2^-9 into the fp32 state, so V~
// enters as a sum of three bf16 terms (24 bits) whose products are exact, the smallest first
// (of each half chunk).
// KV is a new accumulator for every chunk, added to S by an fp32 fma: the tensor cores truncate
// what they accumulate, and a state kept there lost 2e-7 of itself with each chunk of its memory
// (measured: 7e-6 after 4096 tokens at a decay of 1 - 2^-11).  S is rounded to bf16 for O1, P
// for O2: one rounding of an operand each, as the output's own.
//
// Bound: HBM, 2 (d_k + d_v) 2 bytes a token and head: 64 KB a chunk at d = 128, about 2800 cycles
// of an SM's share of 6.5 TB/s.  Next to it is shared memory: at N = 128 a product reads its two
// operands at the full 128 bytes a cycle.  So V~^T and S are A operands from tensor memory, K is
// read as TMA left it, and nothing but P and the outputs is written (with decayed keys as three
// tiles in shared memory a chunk took 7600 cycles).  Passes run beside each other: warps 0-7
// the state, 8-15 V~ (four the first 32 tokens of a chunk, four the others, each as soon as KV has
// read its half), 16-19 P, 20-23 the outputs, 24 and 25 issue (24 G, O1, O2; 25 KV, which waits
// for none of them), 26 loads up to four chunks ahead.
//
// Waits are bounded: a give-up sets the status word, drains what is in flight and ends the CTA.

#include "attn_tc.cuh"
#include "lin_common.cuh"
#include "once.h"
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

// Descriptors of a tile's first k-step; the others lie a constant further on (16-byte units).
__device__ __forceinline__ uint64_t k_base(uint32_t tile) { return sdesc(tile, 16, 1024); }
__host__ __device__ constexpr uint64_t k_step(int ks) {          // K-major, 64 rows
  return (uint64_t)((ks >> 2) * kC * 128 + (ks & 3) * 32) >> 4;
}
__device__ __forceinline__ uint64_t mn_base(uint32_t tile, bool two_panels) {
  return sdesc(tile, two_panels ? kC * 128 : 0, 1024);
}
__host__ __device__ constexpr uint64_t mn_step(int ks) { return (uint64_t)(ks * 2048) >> 4; }

// The passes move data between shared and tensor memory in 8 x 8 matrices, a thread holding two
// neighbouring columns of row lane / 4 (ldmatrix, stmatrix, and the 16-lane shapes of tcgen05.ld
// and .st all agree on it), which transposes without shuffles.
//
// tcgen05.ld of 16 lanes x 16 columns of fp32: x[4 n + 2 h + e] is row lane / 4 + 8 h, column
// 8 n + 2 (lane % 4) + e.
__device__ __forceinline__ void tmem_ld_16x16(uint32_t taddr, float (&v)[8]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}
// tcgen05.st of 16 lanes x 8 columns: r[2 n + h] to row lane / 4 + 8 h, column 4 n + lane % 4.
__device__ __forceinline__ void tmem_st_16x8(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
         "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
         "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void stsm4(uint32_t addr, const float (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};"
               :: "r"(addr), "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]) : "memory");
}
__device__ __forceinline__ void stsm4_t(uint32_t addr, const float (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
               :: "r"(addr), "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]) : "memory");
}

// Where this thread's matrix row of a [64 tokens][DV channels] tile lies, for ldmatrix and
// stmatrix over 16 tokens x 16 channels (matrix i = lane / 8: tokens 8 (i / 2) .., channels
// 8 (i % 2) ..): the first 16 of the warp's 32 channels, and the second 16.
template <int DV>
struct TileRow {
  uint32_t at[2];
  __device__ __forceinline__ TileRow(uint32_t tile, int warp, int lane) {
    const int ch = (warp & 3) * 32 % DV, i = lane >> 3, tok = (i >> 1) * 8 + (lane & 7);
#pragma unroll
    for (int hh = 0; hh < 2; ++hh)
      at[hh] = tile + (uint32_t)((ch >> 6) * kC * 128 + tok * 128 +
                                 (((((ch & 63) >> 3) + 2 * hh + (i & 1)) ^ (lane & 7)) << 4));
  }
};

// The weights of this thread's tokens 16 part + 8 n + 2 (lane % 4) + {0, 1}, for four parts.
struct TokenWeights {
  float2 w[8];
  __device__ __forceinline__ void load(const float* wt, int lane) {
#pragma unroll
    for (int m = 0; m < 8; ++m)
      w[m] = *reinterpret_cast<const float2*>(wt + 8 * m + 2 * (lane & 3));
  }
};

// V~^T of parts p0 .. p0 + NP - 1 (16 tokens each) of a chunk into tensor memory by four warps:
// value channels in the lanes, two tokens to a column; each half chunk has its three bf16 terms
// of 16 columns one after the other.
// The terms are cut off rather than rounded, which leaves 16, 8 and 0 of a float's 24 bits:
// their sum is the float.
template <int NP>
__device__ __forceinline__ void weigh_values(const uint32_t (&row)[2], uint32_t taddr,
                                             const TokenWeights& tw, int p0, float far) {
  const float2 far2 = make_float2(far, far), minus = make_float2(-1.f, -1.f);
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      uint32_t x[4], out[3][4];
      ldsm4_t(row[hh] + (uint32_t)(p0 + p) * 2048, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 w = mul2(tw.w[2 * p + (i >> 1)], far2);
        float2 a = mul2(make_float2(__uint_as_float(x[i] << 16),
                                    __uint_as_float(x[i] & 0xffff0000u)), w);
#pragma unroll
        for (int s = 0; s < 3; ++s) {
          const uint32_t ua = __float_as_uint(a.x), ub = __float_as_uint(a.y);
          out[s][i] = __byte_perm(ua, ub, 0x7632);
          if (s < 2)
            a = fma2(make_float2(__uint_as_float(ua & 0xffff0000u),
                                 __uint_as_float(ub & 0xffff0000u)), minus, a);
        }
      }
#pragma unroll
      for (int s = 0; s < 3; ++s)
        tmem_st_16x8(taddr + ((uint32_t)(16 * hh) << 16) + 48 * ((p0 + p) >> 1) + 16 * s +
                         8 * ((p0 + p) & 1), out[s]);
    }
}

// The share of token half t in KV = V~^T K (A in tensor memory, B the K tile), NH panels of 64
// key channels from panel h on.
template <int NH>
__device__ __forceinline__ void issue_kv(uint32_t d, uint32_t vw, uint32_t k_tile, int t, int h) {
  constexpr uint32_t id = idesc_bf16_mn(128, 64 * NH);
  const uint64_t kb = mn_base(k_tile + h * kC * 128, NH == 2) + mn_step(2) * t;
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      mma_bf16_ta_w(d + 64 * h, vw + 48 * t + 16 * s + 8 * ks, kb + mn_step(ks), id,
                    t > 0 || s < 2 || ks > 0);
}

struct LinMaps {
  CUtensorMap q[kLinMaxJobs], k[kLinMaxJobs], v[kLinMaxJobs], o[kLinMaxJobs];
};

// Weights of the rows of a whole chunk and of the call's ragged last one: a^(L-1-i), where row r
// is token i = r, or L-1-r in a reversed scan.
struct RowTables {
  float wt[2][kC];
};
__device__ __forceinline__ float row_weight(double l2, int rev, int L, int r) {
  return r < L ? (float)decay_pow(l2, rev ? r : L - 1 - r) : 0.f;
}

// ---- first pass: what a segment leaves in the state ---------------------------------------

template <int DK, int DV>
struct SegLayout {
  static constexpr int KT = kC * DK * 2, VT = kC * DV * 2;
  static constexpr int STAGE = KT + VT, STAGES = 6;
  static constexpr int TAB = STAGES * STAGE;
  static constexpr int SMALL = TAB + (int)sizeof(RowTables);
  static constexpr int SMEM = SMALL + 512 + 1024;
  static_assert(SMEM <= 232448, "shared memory");
  // tensor memory: KV and V~ of buffer w
  static constexpr uint32_t KV = 0;                      // + 128 w
  static constexpr uint32_t VW = 256;                    // + 96 w
};
struct SegSmall {
  unsigned long long full[6], empty[6], vw_full[2], kv_done[2], kv_free[2], drained;
  float far[6];                     // of each stage: a^(tokens of the segment after its chunk)
  uint32_t tmem;
  int abort;
};
constexpr int kSegWarps = 16;       // 0-3 sum, 4-7 and 8-11 V~ of every other chunk, 12, 13

template <int DK, int DV>
__global__ void __launch_bounds__(kSegWarps * 32, 1)
lin_segment_tc(const __grid_constant__ LinMaps maps, const LinScan sc, uint32_t spin) {
  using L = SegLayout<DK, DV>;
  constexpr int NS = L::STAGES;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  SegSmall& ss = *reinterpret_cast<SegSmall*>(sm + L::SMALL);
  RowTables& tab = *reinterpret_cast<RowTables*>(sm + L::TAB);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int job = blockIdx.y;
  const int rev = sc.job[job].rev;
  const int p = blockIdx.x % (sc.nseg - 1), bh = blockIdx.x / (sc.nseg - 1);
  const int b = bh / sc.H, h = bh % sc.H;
  const Segment sg = segment(p, rev, sc.T, sc.seg_len, sc.nseg);
  const int nch = (sg.n + kC - 1) / kC;
  const double l2 = log2_decay(sc.decay[h]);
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(mb(ss.full[s]), 1);
      mbar_init(mb(ss.empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(mb(ss.vw_full[s]), 4);
      mbar_init(mb(ss.kv_done[s]), 1);
      mbar_init(mb(ss.kv_free[s]), 4);
    }
    mbar_init(mb(ss.drained), 1);
    ss.abort = 0;
    fence_mbar_init();
  }
  let_next_start();
  if (tid < 2 * kC)
    tab.wt[tid / kC][tid % kC] =
        row_weight(l2, rev, tid < kC ? kC : sg.n - (nch - 1) * kC, tid % kC);
  if (warp == 0) tmem_alloc(&ss.tmem, 512);
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
        tmem_ld32(tb + tl + L::KV + 128 * w + 32 * q, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) S[32 * q + e] += x[e];
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb(ss.kv_free[w]));
    }
    if (ok && v < DV) {
      float* dst = sc.part + (((size_t)job * sc.B * sc.H + bh) * sc.nseg + p + 1) * DV * DK;
#pragma unroll
      for (int e = 0; e < DK / 4; ++e)
        *reinterpret_cast<float4*>(dst + part_at(DV, v, 4 * e)) =
            make_float4(S[4 * e], S[4 * e + 1], S[4 * e + 2], S[4 * e + 3]);
    }
  } else if (warp < 12) {
    fewer_registers<104>();
    // ---- V~ ----------------------------------------------------------------------------------
    const int w = warp < 8 ? 0 : 1;
    const uint32_t tl = (uint32_t)((warp & 3) * 32) << 16;
    TokenWeights tw;
    tw.load(tab.wt[0], lane);
    for (int c = w; c < nch; c += 2) {
      const int s = c % NS;
      if (sg.n - c * kC < kC) tw.load(tab.wt[1], lane);      // the last chunk
      if (!wait(mb(ss.full[s]), (uint32_t)(c / NS) & 1u)) break;
      // the product of chunk c - 2 has read this buffer
      if (c >= 2 && !wait(mb(ss.kv_done[w]), (uint32_t)((c - 2) >> 1) & 1u)) break;
      fence_after_sync();
      const TileRow<DV> row(sb + s * L::STAGE + L::KT, warp, lane);
      weigh_values<4>(row.at, tb + tl + L::VW + 96 * w, tw, 0, ss.far[s]);
      tmem_wait_st();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb(ss.vw_full[w]));
    }
  } else {
    fewer_registers<80>();
    if (warp == 12) {
      for (int c = 0; c < nch; ++c) {
        const int s = c % NS, w = c & 1;
        if (!wait(mb(ss.full[s]), (uint32_t)(c / NS) & 1u)) break;
        if (!wait(mb(ss.vw_full[w]), (uint32_t)(c >> 1) & 1u)) break;
        if (c >= 2 && !wait(mb(ss.kv_free[w]), (uint32_t)((c - 2) >> 1) & 1u)) break;
        fence_after_sync();
        issue_kv<DK / 64>(tb + L::KV + 128 * w, tb + L::VW + 96 * w, sb + s * L::STAGE, 0, 0);
        issue_kv<DK / 64>(tb + L::KV + 128 * w, tb + L::VW + 96 * w, sb + s * L::STAGE, 1, 0);
        mma_commit_w(mb(ss.kv_done[w]));
        mma_commit_w(mb(ss.empty[s]));
      }
      // the products issued here complete before tensor memory is freed
      mma_commit_w(mb(ss.drained));
      mbar_wait(mb(ss.drained), 0, kDrain);
    } else if (warp == 13) {
      int done = 0;
      for (int c = 0; c < nch; ++c) {
        const int s = c % NS;
        if (!wait(mb(ss.empty[s]), ((uint32_t)(c / NS) & 1u) ^ 1u)) break;
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
        for (int c = max(0, done - NS); c < done; ++c)
          mbar_wait(mb(ss.full[c % NS]), (uint32_t)(c / NS) & 1u, kDrain);
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tb, 512);
}

// ---- second pass: the outputs -----------------------------------------------------------------

struct OutTables {
  RowTables rows;
  float fo[4][kC];                  // a^(i+E): [E + 2 ragged]
  float gap[2 * kC];                // [63 + t - j]: a^|t-j| where row t sees row j, else 0
};

template <int DK, int DV>
struct OutLayout {
  static constexpr int KT = kC * DK * 2, VT = kC * DV * 2;
  static constexpr int STAGE = 2 * KT + VT, STAGES = 4;  // q, k, v
  static constexpr int P = STAGES * STAGE;               // bf16 [64 t][64 j], two of them
  static constexpr int O = P + 2 * 8192;                 // outputs on their way out
  static constexpr int TAB = O + VT;
  static constexpr int SMALL = TAB + (int)sizeof(OutTables);
  static constexpr int SMEM = SMALL + 256;      // no room to pad to 1024 bytes by hand
  static_assert(SMEM <= 232448, "shared memory");
  // tensor memory
  static constexpr uint32_t KV = 0;                      // DK columns
  static constexpr uint32_t SB = 128;                    // the state in bf16, DK / 2 columns
  static constexpr uint32_t G = 192;
  static constexpr uint32_t VW = 256;                    // 96 columns
  static constexpr uint32_t O1 = 384, O2 = 448;
};
struct OutSmall {
  unsigned long long full[4], empty[4];
  unsigned long long g_full, p_full[2], vw_full[2], vw_free[2], kv_done[2], kv_free[2], s_ready,
      o1_done, o_full, o_free, drained[2];
  uint32_t tmem;
  int abort;
};
// seven warpgroups: 896 threads of 72 registers at launch, then 2 x 112 + 2 x 56 + 56 + 64 + 48
constexpr int kOutWarps = 28;

template <int DK, int DV>
__global__ void __launch_bounds__(kOutWarps * 32, 1)
lin_out_tc(const __grid_constant__ LinMaps maps, const LinScan sc, uint32_t spin) {
  using L = OutLayout<DK, DV>;
  constexpr int NS = L::STAGES;
  extern __shared__ __align__(1024) unsigned char sm[];
  if ((smem_u32(sm) & 1023u) != 0) {       // the tiles' swizzle needs it
    if (threadIdx.x == 0) atomicOr(sc.status, 1u);
    return;
  }
  OutSmall& os = *reinterpret_cast<OutSmall*>(sm + L::SMALL);
  OutTables& tab = *reinterpret_cast<OutTables*>(sm + L::TAB);
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
    for (int s = 0; s < NS; ++s) {
      mbar_init(mb(os.full[s]), 1);
      mbar_init(mb(os.empty[s]), 2);               // both issuing warps have read the stage
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(mb(os.p_full[s]), 4);
      mbar_init(mb(os.drained[s]), 1);
      mbar_init(mb(os.vw_full[s]), 4);
      mbar_init(mb(os.vw_free[s]), 1);
      mbar_init(mb(os.kv_done[s]), 1);
      mbar_init(mb(os.kv_free[s]), 4);
    }
    mbar_init(mb(os.g_full), 1);
    mbar_init(mb(os.s_ready), 8);
    mbar_init(mb(os.o1_done), 1);
    mbar_init(mb(os.o_full), 1);
    mbar_init(mb(os.o_free), 4);
    os.abort = 0;
    fence_mbar_init();
  }
  {
    const int ragged = sg.n - (nch - 1) * kC;
    const int r = tid % kC, x = tid / kC;          // fourteen rows of 64 threads
    if (x < 2) {
      tab.rows.wt[x][r] = row_weight(l2, rev, x ? ragged : kC, r);
    } else if (x < 6) {
      const int Lc = x >= 4 ? ragged : kC;
      tab.fo[x - 2][r] = (float)decay_pow(l2, (rev ? max(Lc - 1 - r, 0) : r) + (x & 1));
    } else if (x < 8) {
      const int g = (tid - 6 * kC) - (kC - 1);     // t - j
      tab.gap[tid - 6 * kC] = (rev ? g <= 0 : g >= 0) ? (float)decay_pow(l2, rev ? -g : g) : 0.f;
    }
  }
  if (warp == 0) tmem_alloc(&os.tmem, 512);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tb = os.tmem;
  const uint32_t sb = smem_u32(sm);
  const Waits wait{sc.status, &os.abort, spin};
  // chunk c in processing order: its first token in the segment
  auto chunk_at = [&](int c) { return (rev ? nch - 1 - c : c) * kC; };

  if (warp < 8) {
    more_registers<112>();
    // ---- the state: a thread has a row's first or second half ------------------------------
    // (with d_k = 64 the two halves are in one panel of KV, which both wait for)
    constexpr int DH = DK / 2;
    const int v = (warp & 3) * 32 + lane, hf = warp < 4 ? 0 : 1, col = hf * DH;
    const int pn = DK == 128 ? hf : 0;
    const uint32_t tl = (uint32_t)((warp & 3) * 32) << 16;
    // entering: what lin_carry.cu left for this segment, or the call's own state if it is the
    // only one
    float S[DH];
#pragma unroll
    for (int e = 0; e < DH; ++e) S[e] = 0.f;
    const LinJob& jb = sc.job[job];
    if (sc.nseg > 1) {
      wait_for_previous();
      const float* s = sc.part + (((size_t)job * sc.B * sc.H + bh) * sc.nseg + p) * DV * DK;
      if (v < DV) {
#pragma unroll
        for (int e = 0; e < DH / 4; ++e) {
          const float4 y = *reinterpret_cast<const float4*>(s + part_at(DV, v, col + 4 * e));
          S[4 * e] = y.x;
          S[4 * e + 1] = y.y;
          S[4 * e + 2] = y.z;
          S[4 * e + 3] = y.w;
        }
      }
    } else if (v < DV && jb.s_in) {
      const float* s = jb.s_in + (size_t)bh * DV * DK;
      if (jb.s_trans) {
#pragma unroll
        for (int e = 0; e < DH; ++e) S[e] = s[(size_t)(col + e) * DV + v];
      } else {
#pragma unroll
        for (int e = 0; e < DH / 4; ++e) {
          const float4 y = *reinterpret_cast<const float4*>(s + (size_t)v * DK + col + 4 * e);
          S[4 * e] = y.x;
          S[4 * e + 1] = y.y;
          S[4 * e + 2] = y.z;
          S[4 * e + 3] = y.w;
        }
      }
    }
    // a chunk's decay as a pair of floats: its rounding would otherwise be the same in every
    // chunk and add up over a long prompt
    float fh = 0.f, fl = 0.f;
    int steps = -1;
    bool ok = true;
    for (int c = 0; c < nch; ++c) {
      // the bf16 copy, once O1 of the chunk before has read the last one
      if (c > 0 && !(ok = wait(mb(os.o1_done), (uint32_t)(c - 1) & 1u))) break;
      fence_after_sync();
#pragma unroll
      for (int q = 0; q < DH / 32; ++q) {
        uint32_t y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          y[e] = __float_as_uint(pack2(S[32 * q + 2 * e], S[32 * q + 2 * e + 1]));
        tmem_st16(tb + tl + L::SB + col / 2 + 16 * q, y);
      }
      tmem_wait_st();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb(os.s_ready));
      if (c >= nstate) break;
      const int now = min(kC, sg.n - chunk_at(c)) - 1 + (p == 0 && c == 0 ? e0 : 1);
      if (now != steps) {
        const double f = decay_pow(l2, now);
        fh = (float)f;
        fl = (float)(f - (double)fh);
        steps = now;
      }
      const float2 fh2 = make_float2(fh, fh), fl2 = make_float2(fl, fl);
      if (!(ok = wait(mb(os.kv_done[pn]), (uint32_t)c & 1u))) break;
      fence_after_sync();
#pragma unroll
      for (int q = 0; q < DH / 32; ++q) {
        float x[32];
        tmem_ld32(tb + tl + L::KV + col + 32 * q, x);
        tmem_wait_ld();
        if (q == DH / 32 - 1) {
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(mb(os.kv_free[hf]));
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 u = make_float2(S[32 * q + e], S[32 * q + e + 1]);
          const float2 y = fma2(fh2, u, fma2(fl2, u, make_float2(x[e], x[e + 1])));
          S[32 * q + e] = y.x;
          S[32 * q + e + 1] = y.y;
        }
      }
    }
    if (s_out && ok && v < DV) {
      const float f = (float)decay_pow(l2, 1 - e0);
      float* dst = s_out + (size_t)bh * DV * DK + (size_t)v * DK + col;
#pragma unroll
      for (int e = 0; e < DH / 4; ++e)
        reinterpret_cast<float4*>(dst)[e] = make_float4(f * S[4 * e], f * S[4 * e + 1],
                                                        f * S[4 * e + 2], f * S[4 * e + 3]);
    }
  } else if (warp < 16) {
    fewer_registers<56>();
    // ---- V~ ----------------------------------------------------------------------------------
    const uint32_t tl = (uint32_t)((warp & 3) * 32) << 16;
    const int half = warp < 12 ? 0 : 1, p0 = 2 * half;
    TokenWeights tw;
    for (int c = 0; c < nstate; ++c) {
      const int s = c % NS;
      // in the scan's order the ragged chunk comes last, or first and the others after it
      const int ragged = sg.n - chunk_at(c) < kC;
      if (c == 0 || ragged || (rev && c == 1)) tw.load(tab.rows.wt[ragged] + 16 * p0, lane);
      if (!wait(mb(os.full[s]), (uint32_t)(c / NS) & 1u)) break;
      // the products of the chunk before have read this half
      if (c > 0 && !wait(mb(os.vw_free[half]), (uint32_t)(c - 1) & 1u)) break;
      fence_after_sync();
      const TileRow<DV> row(sb + s * L::STAGE + 2 * L::KT, warp, lane);
      weigh_values<2>(row.at, tb + tl + L::VW, tw, p0, 1.f);
      tmem_wait_st();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb(os.vw_full[half]));
    }
  } else if (warp < 20) {
    fewer_registers<56>();
    // ---- P -------------------------------------------------------------------------------------
    // an M = 64 accumulator: row t in lane 32 (t / 16) + t % 16.  This thread's elements and
    // their decays are the same in every chunk
    const int t0 = 16 * (warp & 3) + (lane >> 2), j0 = 2 * (lane & 3);
    const uint32_t tl = (uint32_t)((warp & 3) * 32) << 16;
    float2 g[16];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float* at = tab.gap + kC - 1 + t0 + 8 * hf - 8 * n - j0;
        g[2 * n + hf] = make_float2(at[0], at[-1]);
      }
    // matrix i = lane / 8: columns 8 (i / 2) .., rows 8 (i % 2) ..
    const int tr = 16 * (warp & 3) + (lane & 8) + (lane & 7), n0 = lane >> 4;
    for (int c = 0; c < nch; ++c) {
      if (!wait(mb(os.g_full), (uint32_t)c & 1u)) break;
      fence_after_sync();
      // P's buffer was last read by O2 of chunk c - 2, which came before this G in the pipe
      const uint32_t pt = sb + L::P + (c & 1) * 8192 + tr * 128;
#pragma unroll
      for (int part = 0; part < 4; ++part) {
        float x[8], y[4];
        tmem_ld_16x16(tb + tl + L::G + 16 * part, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 z = mul2(make_float2(x[2 * i], x[2 * i + 1]), g[4 * part + i]);
          y[i] = pack2(z.x, z.y);
        }
        stsm4(pt + (((2 * part + n0) ^ (tr & 7)) << 4), y);
      }
      fence_smem_to_async();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb(os.p_full[c & 1]));
    }
  } else if (warp < 24) {
    fewer_registers<64>();
    // ---- the outputs -----------------------------------------------------------------------
    const uint32_t tl = (uint32_t)((warp & 3) * 32) << 16;
    const TileRow<DV> row(sb + L::O, warp, lane);
    const bool mine = (warp & 3) * 32 < DV;
    bool ok = true;
    for (int c = 0; c < nch; ++c) {
      ok = wait(mb(os.o_full), (uint32_t)c & 1u);
      // the last store has read its tile
      if (tid == 20 * 32) bulk_wait_read_all();
      if (named_bar_or(1, 128, !ok)) break;
      fence_after_sync();
      const int at = chunk_at(c);
      const float* fo = tab.fo[(p == 0 && c == 0 ? e0 : 1) + (sg.n - at < kC ? 2 : 0)];
#pragma unroll
      for (int part = 0; part < 4; ++part) {
        const float2 f0 = *reinterpret_cast<const float2*>(fo + 16 * part + 2 * (lane & 3));
        const float2 f1 = *reinterpret_cast<const float2*>(fo + 16 * part + 8 + 2 * (lane & 3));
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float x[8], y[8], z[4];
          const uint32_t at = tb + tl + ((uint32_t)(16 * hh) << 16) + 16 * part;
          tmem_ld_16x16(at + L::O1, x);
          tmem_ld_16x16(at + L::O2, y);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 u = fma2(make_float2(x[2 * i], x[2 * i + 1]), i < 2 ? f0 : f1,
                                  make_float2(y[2 * i], y[2 * i + 1]));
            z[i] = pack2(u.x, u.y);
          }
          if (mine) stsm4_t(row.at[hh] + part * 2048, z);
        }
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb(os.o_free));
      fence_smem_to_async();
      named_bar(1, 128);
      if (tid == 20 * 32) {
        // rows past the tensor's end are not written
        for (int pn = 0; pn < DV / 64; ++pn)
          tma_store_4d(&maps.o[job], sb + L::O + pn * kC * 128, 64 * pn, h, sg.a + at, b);
        bulk_commit();
      }
    }
    if (tid == 20 * 32) bulk_wait_all();
  } else {
    fewer_registers<48>();
    if (warp == 24) {
      // ---- issuing warp: G, O1, O2 ---------------------------------------------------------------
      constexpr uint32_t id_g = idesc_bf16(64, 64), id_o1 = idesc_bf16(128, 64),
                         id_o2 = idesc_a_mn(idesc_bf16(128, 64));
      auto issue_g = [&](int c) -> bool {
        const uint32_t at = sb + (c % NS) * L::STAGE;
        if (!wait(mb(os.full[c % NS]), (uint32_t)(c / NS) & 1u)) return false;
        fence_after_sync();
        const uint64_t qd = k_base(at), kd = k_base(at + L::KT);
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks)
          mma_bf16_w(tb + L::G, qd + k_step(ks), kd + k_step(ks), id_g, ks > 0);
        mma_commit_w(mb(os.g_full));
        return true;
      };
      bool ok = issue_g(0);
      for (int c = 0; c < nch && ok; ++c) {
        const uint32_t at = sb + (c % NS) * L::STAGE;
        const int w = c & 1;
        // P of this chunk has been formed, so G is free for the next one
        if (!wait(mb(os.p_full[w]), (uint32_t)(c >> 1) & 1u)) break;
        if (c + 1 < nch && !issue_g(c + 1)) break;
        if (c > 0 && !wait(mb(os.o_free), (uint32_t)(c - 1) & 1u)) break;
        fence_after_sync();
        const uint64_t vd = mn_base(at + 2 * L::KT, DV == 128), pd = k_base(sb + L::P + w * 8192);
#pragma unroll
        for (int ks = 0; ks < kC / 16; ++ks)
          mma_bf16_w(tb + L::O2, vd + mn_step(ks), pd + k_step(ks), id_o2, ks > 0);
        if (!wait(mb(os.s_ready), (uint32_t)c & 1u)) break;
        fence_after_sync();
        const uint64_t qd = k_base(at);
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks)
          mma_bf16_ta_w(tb + L::O1, tb + L::SB + 8 * ks, qd + k_step(ks), id_o1, ks > 0);
        mma_commit_w(mb(os.o1_done));
        mma_commit_w(mb(os.o_full));
        mma_commit_w(mb(os.empty[c % NS]));
      }
      // the products issued here complete before tensor memory is freed
      mma_commit_w(mb(os.drained[0]));
      mbar_wait(mb(os.drained[0]), 0, kDrain);
    } else if (warp == 25) {
      // ---- issuing warp: KV ------------------------------------------------------------------------
      for (int c = 0; c < nch; ++c) {
        const int s = c % NS;
        if (c < nstate) {
          if (!wait(mb(os.full[s]), (uint32_t)(c / NS) & 1u)) break;
          // In panels of 64 key channels, each free as soon as its half of the state has taken
          // the chunk before; both panels take a half chunk's V~ before the next, which frees it
          const uint32_t kt = sb + s * L::STAGE + L::KT;
          bool ok = true;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!(ok = ok && wait(mb(os.vw_full[t]), (uint32_t)c & 1u))) break;
#pragma unroll
            for (int h = 0; h < DK / 64; ++h) {
              if (t == 0 && c > 0) {
                if (!(ok = wait(mb(os.kv_free[h]), (uint32_t)(c - 1) & 1u))) break;
                if (DK == 64 && !(ok = wait(mb(os.kv_free[1]), (uint32_t)(c - 1) & 1u))) break;
              }
              fence_after_sync();
              issue_kv<1>(tb + L::KV, tb + L::VW, kt, t, h);
              if (t == 1) mma_commit_w(mb(os.kv_done[h]));
            }
            if (!ok) break;
            mma_commit_w(mb(os.vw_free[t]));
          }
          if (!ok) break;
          mma_commit_w(mb(os.empty[s]));
        } else if (lane == 0) {
          mbar_arrive(mb(os.empty[s]));
        }
      }
      mma_commit_w(mb(os.drained[1]));
      mbar_wait(mb(os.drained[1]), 0, kDrain);
    } else if (warp == 26) {
      // ---- loader -----------------------------------------------------------------------------------
      int done = 0;
      for (int c = 0; c < nch; ++c) {
        const int s = c % NS;
        if (!wait(mb(os.empty[s]), ((uint32_t)(c / NS) & 1u) ^ 1u)) break;
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
        for (int c = max(0, done - NS); c < done; ++c)
          mbar_wait(mb(os.full[c % NS]), (uint32_t)(c / NS) & 1u, kDrain);
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
        !encode_bthd_bf16(&maps.v[j], sc.job[j].v, sc.B, sc.T, sc.H, DV, 64, kC, true) ||
        !encode_bthd_bf16(&maps.o[j], sc.job[j].o, sc.B, sc.T, sc.H, DV, 64, kC, true))
      return cudaErrorInvalidValue;
  const uint32_t spin = attn_spin_limit();
  static std::atomic<unsigned long long> done{0}, done2{0};
  cudaError_t e;
  if (sc.nseg > 1) {
    auto kern = lin_segment_tc<DK, DV>;
    constexpr int smem = SegLayout<DK, DV>::SMEM;
    e = allow_smem(kern, smem, done);
    if (e != cudaSuccess) return e;
    kern<<<dim3((unsigned)(sc.B * sc.H * (sc.nseg - 1)), sc.njobs), kSegWarps * 32, smem, st>>>(
        maps, sc, spin);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_lin_carry(sc, st);
    if (e != cudaSuccess) return e;
  }
  auto kern = lin_out_tc<DK, DV>;
  constexpr int smem = OutLayout<DK, DV>::SMEM;
  e = allow_smem(kern, smem, done2);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(sc.B * sc.H * sc.nseg), sc.njobs);
  if (sc.nseg > 1) return launch_after(kern, grid, kOutWarps * 32, smem, st, maps, sc, spin);
  kern<<<grid, kOutWarps * 32, smem, st>>>(maps, sc, spin);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_tc(const LinScan& sc, cudaStream_t st) {
  if (sc.dk == 128) return sc.dv == 128 ? launch_t<128, 128>(sc, st) : launch_t<128, 64>(sc, st);
  return sc.dv == 128 ? launch_t<64, 128>(sc, st) : launch_t<64, 64>(sc, st);
}

}  // namespace gdr
