// Gradients of sliding-window attention on the tensor cores (sm_100a, tcgen05 + TMA): bf16,
// d = 64, 128.  Mathematics and mask: attn_common.cuh; c = scale log2 e, lse and D = do . o of
// every query are given.  Two kernels, each of which rebuilds the weights:
//
//   dq   a CTA per tile of 128 queries of a head, over key tiles of 64:
//            S = Q K^T,  dP = dO V^T,  dS = 2^(c S - lse) (dP - D),  dQ += dS K
//   dk, dv   a CTA per tile of 128 keys of a key head, over tiles of 64 queries of every head
//        of its group, transposed so that the weights are again an A operand from tensor
//        memory:
//            S^T = K Q^T,  dP^T = V dO^T,  dV += P^T dO,  dK += dS^T Q
//
// Seven products of 128 x 64 x d per tile of 128 x 64 pairs instead of the five that one kernel
// with shared dq sums would need; in exchange no sum crosses CTAs out of order: the results do
// not depend on scheduling.  Bound: the products, 256 cycles each at d = 128; the 64 exponentials
// a thread (512 cycles) run beside them, because two groups of four warps take the tiles in
// turn.  TMEM holds S and dP twice (256 columns) and the sums (dq, or dv and dk: 256); P and dS
// overwrite S and dP as bf16 operands.
//
// P and dS are rounded to bf16, as what they multiply is; the scale is applied to the fp32 sums.
// Where a query sees few keys (up to kFew, or in a prompt of up to 4 kFew + 3 tokens) the rounded o
// inside D weighs as much as these roundings (all three together are 1.5 times the rounding of the
// results), so there P and dS enter as two bf16 terms each, the second in the columns that the first
// leaves free: four or eight more products a step (15 % of the time at a window of 1024 over 4096
// tokens, where it is not done; the errors of dq and dk are 1.1 to 1.2 times the rounding of the
// result with it, 1.5 without, those of dv 1.0 and 1.4).
//
// Key tiles that many queries see are cut (attn_parts.cuh).

#include "attn_parts.cuh"
#include "attn_tc.cuh"
#include "once.h"
#include "tma_host.h"

namespace gdr {
namespace {

using namespace attn;

constexpr int kA = 128;                     // rows of the tile that stays
constexpr int kS = 64;                      // rows of the tiles that stream past
constexpr int kWarpsB = 12;                 // 2 x 4 compute, then issue, load, 2 idle
constexpr int kStages = 3;
constexpr int kFew = 512;

template <int D>
struct BwdLayout {
  static constexpr int BIG = kA * D * 2, SMALL_T = kS * D * 2;
  static constexpr int X = 0, Y = BIG;                   // Q, dO  or  K, V
  static constexpr int ST = 2 * BIG;                     // stages of (K, V) or (Q, dO)
  static constexpr int STAGE = 2 * SMALL_T;
  static constexpr int VEC = ST + kStages * STAGE;       // stages of lse log2 e and D, 64 each
  static constexpr int SMALL = VEC + kStages * 512;
  static constexpr int SMEM = SMALL + 512 + 1024;
  // tensor memory
  static constexpr uint32_t TS = 0;                      // S of buffer w at 128 w, dP 64 after
  static constexpr uint32_t TG = 256;                    // dq, or dv and D after it dk
  static constexpr uint32_t TA = 384;                    // Q, and D / 2 after it dO (dq only)
};

struct BwdSmall {
  unsigned long long big_full, full[kStages], empty[kStages], raw;
  unsigned long long s_full[2], dp_full[2], p_full[2], all_done, drained;
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ uint64_t* mb(unsigned long long& x) {
  return reinterpret_cast<uint64_t*>(&x);
}

__device__ __forceinline__ uint32_t bwd_setup(BwdSmall& s, int warp, int big_arrivals) {
  if (threadIdx.x == 0) {
    mbar_init(mb(s.big_full), big_arrivals);
    mbar_init(mb(s.raw), 1);
    mbar_init(mb(s.all_done), 1);
    mbar_init(mb(s.drained), 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(mb(s.full[i]), 1);
      mbar_init(mb(s.empty[i]), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(mb(s.s_full[w]), 1);
      mbar_init(mb(s.dp_full[w]), 1);
      mbar_init(mb(s.p_full[w]), 4);
    }
    s.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&s.tmem, 512);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  return s.tmem;
}

// Loads one stage: tiles (x, y) of kS rows from row r0 of head h; rows at and past `limit` of
// what the reduction runs over are zeroed (limit < 0: nothing to hide).  vec: lse and D of the
// rows, when they stream.  Returns false after a give-up.
template <int D>
__device__ __forceinline__ bool load_stage(const CUtensorMap* mx, const CUtensorMap* my,
                                           unsigned char* sm, BwdSmall& bs, int s, int h, int r0,
                                           int b, int limit, uint32_t& nraw, const Waits& wait,
                                           int lane) {
  using L = BwdLayout<D>;
  const bool raw = limit >= 0 && r0 + kS > limit;
  uint64_t* bar = raw ? mb(bs.raw) : mb(bs.full[s]);
  const uint32_t at = smem_u32(sm) + L::ST + s * L::STAGE;
  if (lane == 0) {
    mbar_expect_tx(bar, L::STAGE);
    for (int pn = 0; pn < D / 64; ++pn) {
      tma_load_4d(at + pn * kS * 128, mx, 64 * pn, h, r0, b, bar);
      tma_load_4d(at + L::SMALL_T + pn * kS * 128, my, 64 * pn, h, r0, b, bar);
    }
  }
  if (!raw) return true;
  const bool ok = wait(bar, nraw & 1u);
  if (!ok) mbar_wait(bar, nraw & 1u, kDrain);
  ++nraw;
  zero_rows<D>(sm + L::ST + s * L::STAGE, kS, max(0, limit - r0), lane);
  zero_rows<D>(sm + L::ST + s * L::STAGE + L::SMALL_T, kS, max(0, limit - r0), lane);
  if (lane == 0) mbar_arrive(mb(bs.full[s]));
  return ok;
}

// Copies in flight land before the CTA leaves (`done` stages were loaded).
__device__ __forceinline__ void drain_loads(BwdSmall& bs, int done) {
  for (int y = max(0, done - kStages); y < done; ++y)
    mbar_wait(mb(bs.full[y % kStages]), (uint32_t)(y / kStages) & 1u, kDrain);
}

// The issuing warp of both kernels over n steps.  The tile that stays is an A operand in shared
// memory (K, V for dv and dk), or in tensor memory where that has room for it (Q, dO for dq): at
// N = 64 a product with both operands in shared memory takes 49 cycles, bound by its reads, one
// with A in tensor memory 33.
template <int D, bool DKV, bool FINE>
__device__ __forceinline__ void issue_steps(uint32_t sb, uint32_t tb, BwdSmall& bs, int n,
                                            const Waits& wait) {
  using L = BwdLayout<D>;
  constexpr uint32_t id_s = idesc_bf16(kA, kS), id_g = idesc_bf16_mn(kA, D);
  bool ok = n == 0 || wait(mb(bs.big_full), 0);
  for (int y = 0; y <= n && ok; ++y) {
    if (y < n) {
      const int s = y % kStages, w = y & 1;
      if (!(ok = wait(mb(bs.full[s]), (uint32_t)(y / kStages) & 1u))) break;
      fence_after_sync();
      const uint32_t at = sb + L::ST + s * L::STAGE;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        if (DKV)
          mma_bf16_w(tb + L::TS + 128 * w, kmajor(sb + L::X, kA, ks), kmajor(at, kS, ks), id_s,
                     ks > 0);
        else
          mma_bf16_ta_w(tb + L::TS + 128 * w, tb + L::TA + 8 * ks, kmajor(at, kS, ks), id_s,
                        ks > 0);
      }
      mma_commit_w(mb(bs.s_full[w]));
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        if (DKV)
          mma_bf16_w(tb + L::TS + 128 * w + 64, kmajor(sb + L::Y, kA, ks),
                     kmajor(at + L::SMALL_T, kS, ks), id_s, ks > 0);
        else
          mma_bf16_ta_w(tb + L::TS + 128 * w + 64, tb + L::TA + D / 2 + 8 * ks,
                        kmajor(at + L::SMALL_T, kS, ks), id_s, ks > 0);
      }
      mma_commit_w(mb(bs.dp_full[w]));
    }
    if (y > 0) {
      const int z = y - 1, s = z % kStages, w = z & 1;
      if (!(ok = wait(mb(bs.p_full[w]), (uint32_t)(z >> 1) & 1u))) break;
      fence_after_sync();
      const uint32_t at = sb + L::ST + s * L::STAGE;
      if (DKV) {
#pragma unroll
        for (int ks = 0; ks < (FINE ? 2 : 1) * kS / 16; ++ks)
          mma_bf16_ta_w(tb + L::TG, tb + L::TS + 128 * w + 8 * ks,
                        mnmajor(at + L::SMALL_T, kS, ks % (kS / 16)), id_g, z > 0 || ks > 0);
      }
#pragma unroll
      for (int ks = 0; ks < (FINE ? 2 : 1) * kS / 16; ++ks)
        mma_bf16_ta_w(tb + L::TG + (DKV ? D : 0), tb + L::TS + 128 * w + 64 + 8 * ks,
                      mnmajor(at, kS, ks % (kS / 16)), id_g, z > 0 || ks > 0);
      mma_commit_w(mb(bs.empty[s]));
    }
  }
  if (ok) mma_commit_w(mb(bs.all_done));
  // the products issued here complete before tensor memory is freed
  mma_commit_w(mb(bs.drained));
  mbar_wait(mb(bs.drained), 0, kDrain);
}

// 64 weights of a TMEM lane as bf16 pairs, with FINE what the rounding cut off in 32 more columns.
template <bool FINE>
__device__ __forceinline__ void put_weights(uint32_t taddr, const float (&x)[kS]) {
  float pk[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) pk[e] = pack2(x[2 * e], x[2 * e + 1]);
  tmem_st32(taddr, pk);
  if (FINE) {
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const uint32_t u = __float_as_uint(pk[e]);
      pk[e] = pack2(x[2 * e] - __uint_as_float(u << 16),
                    x[2 * e + 1] - __uint_as_float(u & 0xffff0000u));
    }
    tmem_st32(taddr + 32, pk);
  }
}

// D columns of a TMEM lane times f, as bf16, to dst (16-byte aligned); zeros when !have.
template <int D>
__device__ __forceinline__ void store_row(uint32_t taddr, float f, bool have, bool write,
                                          __nv_bfloat16* dst) {
#pragma unroll
  for (int q = 0; q < D / 32; ++q) {
    float o[32];
    if (have) {
      tmem_ld32(taddr + 32 * q, o);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = 0.f;
    }
    if (write) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        reinterpret_cast<float4*>(dst + 32 * q)[e] =
            make_float4(pack2(o[8 * e] * f, o[8 * e + 1] * f),
                        pack2(o[8 * e + 2] * f, o[8 * e + 3] * f),
                        pack2(o[8 * e + 4] * f, o[8 * e + 5] * f),
                        pack2(o[8 * e + 6] * f, o[8 * e + 7] * f));
    }
  }
}

template <int D, bool FINE>
__global__ void __launch_bounds__(kWarpsB * 32, 1)
attn_dq_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
           const AttnGradArgs a, uint32_t spin) {
  using L = BwdLayout<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  BwdSmall& bs = *reinterpret_cast<BwdSmall*>(sm + L::SMALL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttnArgs& f = a.f;
  const int nq = (f.Tq + kA - 1) / kA;
  const int h = blockIdx.x % f.Hq;
  const int b = (blockIdx.x / f.Hq) % f.B;
  const int i0 = (nq - 1 - (int)(blockIdx.x / ((unsigned)f.Hq * f.B))) * kA;
  const int hk = h / (f.Hq / f.Hkv);
  const Mask m = make_mask(f.lengths, b, f.Tq, f.Tk, f.window, f.sinks);
  const KeyTiles kt = key_tiles<kS>(m, i0, min(i0 + kA, f.Tq) - 1);
  const int n = kt.count();
  const uint32_t tb = bwd_setup(bs, warp, 8);
  const uint32_t sb = smem_u32(sm);
  const Waits wait{f.status, &bs.abort, spin};

  if (warp < 8) {
    more_registers<208>();
    const int w = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tl = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tb + tl + L::TS + 128 * w;
    const int i = i0 + row, p = m.off + i;
    const float c = f.scale * kLog2e;
    {
      // the query's row into its TMEM lane: q by the first group, do by the second
      const uint4* src = reinterpret_cast<const uint4*>((const __nv_bfloat16*)(w ? a.dO : f.q) +
                                                        (((size_t)b * f.Tq + i) * f.Hq + h) * D);
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        float x[32];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          reinterpret_cast<uint4*>(x)[e] = i < f.Tq ? src[8 * q + e] : make_uint4(0, 0, 0, 0);
        tmem_st32(tb + tl + L::TA + D / 2 * w + 32 * q, x);
      }
      tmem_wait_st();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb(bs.big_full));
    }
    const size_t at = ((size_t)b * f.Hq + h) * f.Tq + i;
    const float nl = i < f.Tq ? -f.lse[at] * kLog2e : 0.f;
    const float nd = i < f.Tq ? -a.delta[at] : 0.f;
    const float2 c2 = make_float2(c, c), nl2 = make_float2(nl, nl), nd2 = make_float2(nd, nd);
    bool ok = true;
    for (int y = w; y < n; y += 2) {
      const int j0 = kt.tile(y) * kS;
      const uint32_t par = (uint32_t)(y >> 1) & 1u;
      if (!(ok = wait(mb(bs.s_full[w]), par))) break;
      fence_after_sync();
      float s[kS], g[kS];
      tmem_ld32(tS, reinterpret_cast<float(&)[32]>(s[0]));
      tmem_ld32(tS + 32, reinterpret_cast<float(&)[32]>(s[32]));
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < kS; e += 2) {
        const float2 x = fma2(make_float2(s[e], s[e + 1]), c2, nl2);
        s[e] = ex2(x.x);
        s[e + 1] = ex2(x.y);
      }
      if (!(ok = wait(mb(bs.dp_full[w]), par))) break;
      fence_after_sync();
      tmem_ld32(tS + 64, reinterpret_cast<float(&)[32]>(g[0]));
      tmem_ld32(tS + 96, reinterpret_cast<float(&)[32]>(g[32]));
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < kS; e += 2) {
        const float2 x = mul2(make_float2(s[e], s[e + 1]),
                              add2(make_float2(g[e], g[e + 1]), nd2));
        g[e] = x.x;
        g[e + 1] = x.y;
      }
      if (!all_visible(m, m.off + i0, m.off + i0 + kA - 1, j0, j0 + kS - 1))
        hide(g, row_cols(m, p, j0), 0.f);
      put_weights<FINE>(tS + 64, g);
      tmem_wait_st();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb(bs.p_full[w]));
    }
    if (ok && n > 0) ok = wait(mb(bs.all_done), 0);
    if (ok && w == 0) {
      fence_after_sync();
      store_row<D>(tb + tl + L::TG, f.scale, n > 0, i < f.Tq,
                   (__nv_bfloat16*)a.dq + (((size_t)b * f.Tq + i) * f.Hq + h) * D);
    }
  } else {
    fewer_registers<80>();
    if (warp == 8) {
      issue_steps<D, false, FINE>(sb, tb, bs, n, wait);
    } else if (warp == 9) {
      const int limit = m.len < f.Tk ? m.len : -1;
      uint32_t nraw = 0;
      int done = 0;
      for (int y = 0; y < n; ++y) {
        const int s = y % kStages;
        if (!wait(mb(bs.empty[s]), ((uint32_t)(y / kStages) & 1u) ^ 1u)) break;
        done = y + 1;
        if (!load_stage<D>(&tm_k, &tm_v, sm, bs, s, hk, kt.tile(y) * kS, b, limit, nraw, wait,
                           lane))
          break;
      }
      if (lane == 0) drain_loads(bs, done);
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tb, 512);
  // its blocks start as those of the kernel before (dk, dv: nothing they need) leave their SMs;
  // this one is not over before that one
  wait_for_previous();
}

template <int D, bool FINE>
__global__ void __launch_bounds__(kWarpsB * 32, 1)
attn_dkv_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
            const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
            const AttnGradArgs a, const Parts parts, uint32_t spin) {
  using L = BwdLayout<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  BwdSmall& bs = *reinterpret_cast<BwdSmall*>(sm + L::SMALL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttnArgs& f = a.f;
  // the first key tiles, which the most queries see, start first
  const int bh = blockIdx.x % (f.B * f.Hkv), item = blockIdx.x / (f.B * f.Hkv);
  const int b = bh / f.Hkv, hk = bh % f.Hkv, G = f.Hq / f.Hkv;
  int tile, part;
  parts.locate(item, tile, part);
  const int j0 = tile * kA;
  const Mask m = make_mask(f.lengths, b, f.Tq, f.Tk, f.window, f.sinks);
  int lo64, nt;
  tile_steps<kA, kS>(m, j0, f.Tk, f.Tq, lo64, nt);
  const int used = parts.used(G * nt, tile);
  let_next_start();
  if (part >= used) return;
  const int per = (G * nt + used - 1) / used;
  const int y0 = part * per, n = max(0, min(per, G * nt - y0));
  const uint32_t tb = bwd_setup(bs, warp, 1);
  const uint32_t sb = smem_u32(sm);
  const Waits wait{f.status, &bs.abort, spin};

  if (warp < 8) {
    more_registers<208>();
    const int w = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tl = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tb + tl + L::TS + 128 * w;
    const int j = j0 + row;
    const float c = f.scale * kLog2e;
    const float2 c2 = make_float2(c, c);
    bool ok = true;
    for (int y = w; y < n; y += 2) {
      const int i0 = (lo64 + (y0 + y) % nt) * kS, p0 = m.off + i0;
      const uint32_t par = (uint32_t)(y >> 1) & 1u;
      const float* vec = reinterpret_cast<const float*>(sm + L::VEC + (y % kStages) * 512);
      // the loader's lse and D, then the scores
      if (!(ok = wait(mb(bs.full[y % kStages]), (uint32_t)(y / kStages) & 1u))) break;
      if (!(ok = wait(mb(bs.s_full[w]), par))) break;
      fence_after_sync();
      float s[kS], g[kS];
      tmem_ld32(tS, reinterpret_cast<float(&)[32]>(s[0]));
      tmem_ld32(tS + 32, reinterpret_cast<float(&)[32]>(s[32]));
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < kS; e += 4) {
        const float4 l = *reinterpret_cast<const float4*>(vec + e);
        const float2 x = fma2(make_float2(s[e], s[e + 1]), c2, make_float2(l.x, l.y));
        const float2 z = fma2(make_float2(s[e + 2], s[e + 3]), c2, make_float2(l.z, l.w));
        s[e] = ex2(x.x);
        s[e + 1] = ex2(x.y);
        s[e + 2] = ex2(z.x);
        s[e + 3] = ex2(z.y);
      }
      // this key's queries as a range of columns
      const bool whole = all_visible(m, p0, p0 + kS - 1, j0, j0 + kA - 1);
      RowCols rc;
      if (!whole) {
        rc = col_rows(m, j, p0);
        hide(s, rc, 0.f);
      }
      put_weights<FINE>(tS, s);
      if (!(ok = wait(mb(bs.dp_full[w]), par))) break;
      fence_after_sync();
      tmem_ld32(tS + 64, reinterpret_cast<float(&)[32]>(g[0]));
      tmem_ld32(tS + 96, reinterpret_cast<float(&)[32]>(g[32]));
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < kS; e += 4) {
        const float4 d = *reinterpret_cast<const float4*>(vec + kS + e);
        const float2 x = mul2(make_float2(s[e], s[e + 1]),
                              add2(make_float2(g[e], g[e + 1]), make_float2(d.x, d.y)));
        const float2 z = mul2(make_float2(s[e + 2], s[e + 3]),
                              add2(make_float2(g[e + 2], g[e + 3]), make_float2(d.z, d.w)));
        g[e] = x.x;
        g[e + 1] = x.y;
        g[e + 2] = z.x;
        g[e + 3] = z.y;
      }
      if (!whole) hide(g, rc, 0.f);     // 0 times what a hidden query holds is not always 0
      put_weights<FINE>(tS + 64, g);
      tmem_wait_st();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(mb(bs.p_full[w]));
    }
    if (ok && n > 0) ok = wait(mb(bs.all_done), 0);
    if (ok) {
      fence_after_sync();
      // warps 0-3: dv; warps 4-7: dk
      const float scale = w ? f.scale : 1.f;
      const uint32_t tg = tb + tl + L::TG + (w ? D : 0);
      if (used == 1) {
        store_row<D>(tg, scale, n > 0, j < f.Tk,
                     (__nv_bfloat16*)(w ? a.dk : a.dv) +
                         (((size_t)b * f.Tk + j) * f.Hkv + hk) * D);
      } else {
        float* dst = a.part + part_at(f, kA, D, item, bh, w, row, 0);
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          float o[32];
          if (n > 0) {
            tmem_ld32(tg + 32 * q, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            reinterpret_cast<float4*>(dst + (size_t)(4 * q + (e >> 1)) * kA * 8)[e & 1] =
                n > 0 ? make_float4(o[4 * e] * scale, o[4 * e + 1] * scale, o[4 * e + 2] * scale,
                                    o[4 * e + 3] * scale)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    }
  } else {
    fewer_registers<80>();
    if (warp == 8) {
      issue_steps<D, true, FINE>(sb, tb, bs, n, wait);
    } else if (warp == 9 && n > 0) {
      if (lane == 0) {
        mbar_expect_tx(mb(bs.big_full), 2 * L::BIG);
        for (int pn = 0; pn < D / 64; ++pn) {
          tma_load_4d(sb + L::X + pn * kA * 128, &tm_k, 64 * pn, hk, j0, b, mb(bs.big_full));
          tma_load_4d(sb + L::Y + pn * kA * 128, &tm_v, 64 * pn, hk, j0, b, mb(bs.big_full));
        }
      }
      const int limit = m.len < f.Tk ? max(0, m.len - m.off) : -1;
      uint32_t nraw = 0;
      int done = 0;
      for (int y = 0; y < n; ++y) {
        const int s = y % kStages;
        const int h = hk * G + (y0 + y) / nt, i0 = (lo64 + (y0 + y) % nt) * kS;
        // this step's lse and D, read before the wait for the stage
        float v[4];
        const size_t at = ((size_t)b * f.Hq + h) * f.Tq + i0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool in = i0 + lane + 32 * e < f.Tq;
          v[e] = in ? -f.lse[at + lane + 32 * e] * kLog2e : 0.f;
          v[2 + e] = in ? -a.delta[at + lane + 32 * e] : 0.f;
        }
        if (!wait(mb(bs.empty[s]), ((uint32_t)(y / kStages) & 1u) ^ 1u)) break;
        float* vec = reinterpret_cast<float*>(sm + L::VEC + s * 512);
#pragma unroll
        for (int e = 0; e < 4; ++e) vec[lane + 32 * e] = v[e];
        __syncwarp();
        done = y + 1;
        if (!load_stage<D>(&tm_q, &tm_do, sm, bs, s, h, i0, b, limit, nraw, wait, lane)) break;
      }
      if (lane == 0) {
        mbar_wait(mb(bs.big_full), 0, kDrain);
        drain_loads(bs, done);
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tb, 512);
}

template <int D, bool FINE>
cudaError_t launch_t(const AttnGradArgs& a, cudaStream_t st) {
  using L = BwdLayout<D>;
  const AttnArgs& f = a.f;
  CUtensorMap kb, vb, qs, ds, ks, vs;      // tiles that stay, tiles that stream
  if (!encode_bthd_bf16(&kb, f.k, f.B, f.Tk, f.Hkv, D, 64, kA, true) ||
      !encode_bthd_bf16(&vb, f.v, f.B, f.Tk, f.Hkv, D, 64, kA, true) ||
      !encode_bthd_bf16(&qs, f.q, f.B, f.Tq, f.Hq, D, 64, kS, true) ||
      !encode_bthd_bf16(&ds, a.dO, f.B, f.Tq, f.Hq, D, 64, kS, true) ||
      !encode_bthd_bf16(&ks, f.k, f.B, f.Tk, f.Hkv, D, 64, kS, true) ||
      !encode_bthd_bf16(&vs, f.v, f.B, f.Tk, f.Hkv, D, 64, kS, true))
    return cudaErrorInvalidValue;
  auto kq = attn_dq_tc<D, FINE>;
  auto kk = attn_dkv_tc<D, FINE>;
  static std::atomic<unsigned long long> done{0}, done2{0};
  cudaError_t e = allow_smem(kq, L::SMEM, done);
  if (e == cudaSuccess)
    e = allow_smem(kk, L::SMEM, done2);
  if (e != cudaSuccess) return e;
  const uint32_t spin = attn_spin_limit();
  const Parts p = plan_parts<kA, kS>(f, 148);
  const unsigned bh = (unsigned)(f.B * f.Hkv);
  kk<<<(unsigned)p.items() * bh, kWarpsB * 32, L::SMEM, st>>>(kb, vb, qs, ds, a, p, spin);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_after(kq, dim3((unsigned)((f.Tq + kA - 1) / kA * f.Hq * f.B)), kWarpsB * 32, L::SMEM,
                   st, ks, vs, a, spin);
  if (e != cudaSuccess) return e;
  return launch_dkv_join<__nv_bfloat16, D, kA, kS>(a, p, st);
}

}  // namespace

// Workspace of the parts' sums (0 when no tile is cut).
size_t attn_backward_tc_bytes(const AttnArgs& f) {
  return part_bytes(f, kA, plan_parts<kA, kS>(f, 148));
}

cudaError_t launch_attn_backward_tc(const AttnGradArgs& a, cudaStream_t st) {
  // The window bounds what every query sees; however wide it is, the first queries of a prompt see
  // few keys, which shows up to about 2048 tokens.  (Lengths lie on the device and do not count.)
  long seen = a.f.Tk / 4;
  if (a.f.window && seen > (long)a.f.window + a.f.sinks) seen = (long)a.f.window + a.f.sinks;
  if (seen <= kFew) return a.f.d == 64 ? launch_t<64, true>(a, st) : launch_t<128, true>(a, st);
  return a.f.d == 64 ? launch_t<64, false>(a, st) : launch_t<128, false>(a, st);
}

}  // namespace gdr
