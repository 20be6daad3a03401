// Sliding-window attention on the tensor cores (sm_100a, tcgen05 + TMA): bf16, d = 64, 128.
//
// Mathematics and mask: attn_common.cuh.  One CTA takes two tiles of 128 queries of a head
// (A and B) over the key tiles of 128 that either of them sees, in one pass with the running
// maximum m and sum l of the softmax:
//
//     S = Q K^T,  P = 2^(c S - c m),  O += P V,  l += rows of P        (c = scale log2 e)
//
// Bound: a pair of tiles takes 4 d 128^2 flops on the tensor cores and 128^2 exponentials, at
// 4096 multiply-adds and 16 exponentials a cycle 1024 cycles of either (d = 128), so both must
// run all the time: while the four warps of tile A form P the tensor cores run tile B's
// products, and the other way round.  Roles: warps 0-3 tile A, warps 4-7 tile B (a thread owns
// a query: its scores are a TMEM lane, so no row statistic crosses threads), warp 8 issues the
// products, warp 9 loads.  S_A, S_B, O_A, O_B fill the 512 TMEM columns; P overwrites the first
// half of S as the bf16 A operand of P V, read from tensor memory.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since the last time (the
// weights then stay below 2^8, far from bf16's range), which after the first key tiles is rare.
// P is rounded to bf16, as the values it weighs are; l adds the unrounded weights.
//
// Few queries over many keys (a short piece of a long prompt) leave SMs without a pair of tiles.
// There the key tiles of a pair are cut into parts, one CTA each, which leave their O, m and l
// in the workspace in fp32, and a second kernel joins them:
//
//     m = max m_p,   l = sum 2^(m_p - m) l_p,   o = sum 2^(m_p - m) O_p / l
//
// (16 queries over 8192 keys, 32 heads of d = 128: 38 us, 127 with one CTA to a pair; 3 x 500
// queries at a window of 1000, 12 heads of d = 64: 22 us and 30.)
//
// Waits are bounded: a give-up sets the status word, drains what is in flight and ends the CTA.

#include "attn_tc.cuh"
#include "once.h"
#include "tma_host.h"

namespace gdr {
namespace {

using namespace attn;

constexpr int kT = 128;                     // queries and keys of a tile
// three warpgroups: 384 threads of 168 registers at launch, then 2 x 128 x 208 + 128 x 80
constexpr int kWarpsF = 12;
constexpr int kSMs = 148, kLeast = 3;       // key tiles of a part
constexpr float kGrow = 8.f;                // log2 of how far a row's weights may grow
constexpr float kLarge = 268435456.f;       // 2^28: the rounding of a base past it may exceed 16

template <int D>
struct FwdLayout {
  static constexpr int TILE = kT * D * 2;
  static constexpr int STAGES = 2;
  static constexpr int Q = 0;                          // tiles A, B
  static constexpr int K = 2 * TILE;
  static constexpr int V = K + STAGES * TILE;
  static constexpr int SMALL = V + STAGES * TILE;
  static constexpr int SMEM = SMALL + 512 + 1024;      // + alignment
  static constexpr uint32_t TS = 0;                    // S of tile w at TS + 128 w
  static constexpr uint32_t TO = 256;                  // O of tile w at TO + D w
};

struct FwdSmall {
  unsigned long long q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], v_raw;
  unsigned long long s_full[2], p_full[2], o_done[2], drained;
  uint32_t tmem;
  int abort;
};

// The key tiles of the pair (of one of `parts` equal parts of them), and which of them each tile
// of queries sees.
struct PairTiles {
  KeyTiles t[2];
  int nsink, lo, first, n;
  __device__ __forceinline__ int tile(int x) const {
    return x + first < nsink ? x + first : lo + x + first - nsink;
  }
};
__device__ __forceinline__ PairTiles pair_tiles(const Mask& m, int i0, int Tq, int part,
                                                int parts) {
  PairTiles p;
  p.t[0] = key_tiles<kT>(m, i0, min(i0 + kT, Tq) - 1);
  p.t[1] = i0 + kT < Tq ? key_tiles<kT>(m, i0 + kT, min(i0 + 2 * kT, Tq) - 1) : KeyTiles{0, 0, 0};
  const KeyTiles& f = p.t[p.t[0].nwin > 0 ? 0 : 1];     // the earlier one that sees anything
  p.lo = f.lo;
  p.nsink = f.nsink;
  const int hi = max(p.t[0].nwin ? p.t[0].lo + p.t[0].nwin : 0,
                     p.t[1].nwin ? p.t[1].lo + p.t[1].nwin : 0);
  const int all = hi > 0 ? p.nsink + hi - p.lo : 0;
  const int per = (all + parts - 1) / parts;
  p.first = part * per;
  p.n = max(0, min(per, all - p.first));
  return p;
}

// A row whose scores are so large that the rounding of its base c m, which stays in its exponents,
// may have taken the weights out of range: once more by the whole warp, in fp32 from global memory,
// the differences of scores formed first.  That happens past scores of 2^28 / log2 e only.  (8192
// tokens, 32 heads: 434 us, 428 without this code and NaN for such rows; 437 to 447 with the
// rounding taken off in the loop.)
// i: the query; thread `owner` has its lane of O at tO.  Returns (c m, l) to all.
template <int D>
__device__ __forceinline__ float2 redo_row(const AttnArgs& a, const Mask& m, const PairTiles& pt,
                                           int w, int b, int h, int i, int owner, uint32_t tO) {
  using T = __nv_bfloat16;
  const int lane = threadIdx.x & 31;
  const float c = a.scale * kLog2e;
  const size_t step = (size_t)a.Hkv * D;
  const size_t kv = (size_t)b * a.Tk * step + (size_t)(h / (a.Hq / a.Hkv)) * D;
  const T* q = (const T*)a.q + (((size_t)b * a.Tq + i) * a.Hq + h) * D;
  auto score = [&](int j, bool sees) {            // each lane its own key
    float s = -INFINITY;
    if (sees) {
      const T* k = (const T*)a.k + kv + j * step;
      s = 0.f;
#pragma unroll 1
      for (int e = 0; e < D; ++e) s = fmaf(Elem<T>::load(q + e), Elem<T>::load(k + e), s);
    }
    return s;
  };
  float top = -INFINITY, l = 0.f, o[D / 32] = {};
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int x = 0; x < pt.n; ++x) {
      const int tl = pt.tile(x);
      if (!(w ? pt.t[1] : pt.t[0]).has(tl)) continue;
      const RowCols rc = row_cols(m, m.off + i, tl * kT);
#pragma unroll 1
      for (int j0 = 0; j0 < kT; j0 += 32) {
        const float s = score(tl * kT + j0 + lane, rc.sees(j0 + lane));
        if (pass == 0) {
          top = fmaxf(top, s);
          continue;
        }
        const float p = s == -INFINITY ? 0.f : ex2((s - top) * c);
        l += p;
#pragma unroll 1
        for (int e = 0; e < 32; ++e) {
          const float pe = __shfl_sync(0xffffffffu, p, e);
          if (pe == 0.f) continue;                // (hidden keys are not read)
          const T* v = (const T*)a.v + kv + (tl * kT + j0 + e) * step;
#pragma unroll
          for (int u = 0; u < D / 32; ++u) o[u] = fmaf(pe, Elem<T>::load(v + 32 * u + lane), o[u]);
        }
      }
    }
    if (pass == 0) {
#pragma unroll
      for (int f = 16; f; f >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, f));
    }
  }
#pragma unroll
  for (int f = 16; f; f >>= 1) l += __shfl_xor_sync(0xffffffffu, l, f);
#pragma unroll
  for (int u = 0; u < D / 32; ++u) {
    float t[32];
    tmem_ld32(tO + 32 * u, t);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float y = __shfl_sync(0xffffffffu, o[u], e);
      if (lane == owner) t[e] = y;
    }
    tmem_st32(tO + 32 * u, t);
  }
  tmem_wait_st();
  return make_float2(top * c, l);
}

template <int D, bool PARTS>
__global__ void __launch_bounds__(kWarpsF * 32, 1)
attn_forward_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const AttnArgs a,
                int nparts, uint32_t spin) {
  using L = FwdLayout<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  FwdSmall& fs = *reinterpret_cast<FwdSmall*>(sm + L::SMALL);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // heads run fastest so that the CTAs in flight share keys; the last queries, which see the
  // most keys when there is no window, start first
  const int npair = (a.Tq + 2 * kT - 1) / (2 * kT);
  const int h = blockIdx.x % a.Hq;
  const int b = (blockIdx.x / a.Hq) % a.B;
  const int parts = PARTS ? nparts : 1;
  const unsigned rest = blockIdx.x / ((unsigned)a.Hq * a.B);
  const int part = PARTS ? rest % parts : 0;
  const int pr = npair - 1 - (int)(rest / parts);
  const int hk = h / (a.Hq / a.Hkv);
  const int i0 = pr * 2 * kT;
  const Mask m = make_mask(a.lengths, b, a.Tq, a.Tk, a.window, a.sinks);
  const PairTiles pt = pair_tiles(m, i0, a.Tq, part, parts);

  auto bar = [](unsigned long long& x) { return reinterpret_cast<uint64_t*>(&x); };
  if (tid == 0) {
    mbar_init(bar(fs.q_full), 1);
    mbar_init(bar(fs.v_raw), 1);
    mbar_init(bar(fs.drained), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(fs.k_full[s]), 1);
      mbar_init(bar(fs.k_empty[s]), 1);
      mbar_init(bar(fs.v_full[s]), 1);
      mbar_init(bar(fs.v_empty[s]), 1);
      mbar_init(bar(fs.s_full[s]), 1);
      mbar_init(bar(fs.p_full[s]), 4);
      mbar_init(bar(fs.o_done[s]), 1);
    }
    fs.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&fs.tmem, 512);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tb = fs.tmem;
  const uint32_t sb = smem_u32(sm);
  const Waits wait{a.status, &fs.abort, spin};

  if (warp < 8) {
    more_registers<208>();
    // ---- softmax of tile w: thread = query ---------------------------------------------------
    const int w = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t tl0 = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tb + tl0 + L::TS + 128 * w, tO = tb + tl0 + L::TO + D * w;
    const int iw = i0 + w * kT, i = iw + row;
    const int p = m.off + i;
    const float c = a.scale * kLog2e;
    const KeyTiles mine = w ? pt.t[1] : pt.t[0];
    float mref = -INFINITY;                 // the maximum (of q.k) the weights refer to
    float2 l2 = make_float2(0.f, 0.f);
    uint32_t ns = 0;                        // score tiles taken
    bool ok = true;
    for (int x = 0; x < pt.n; ++x) {
      const int tl = pt.tile(x), j0 = tl * kT;
      if (!mine.has(tl)) continue;
      if (!(ok = wait(bar(fs.s_full[w]), ns & 1u))) break;
      fence_after_sync();
      float s[kT];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        tmem_ld32(tS + 32 * q, reinterpret_cast<float(&)[32]>(s[32 * q]));
      tmem_wait_ld();
      if (!all_visible(m, m.off + iw, m.off + iw + kT - 1, j0, j0 + kT - 1))
        hide(s, row_cols(m, p, j0), -INFINITY);
      float t0 = s[0], t1 = s[1], t2 = s[2], t3 = s[3];
#pragma unroll
      for (int q = 4; q < kT - 4; q += 8) {
        t0 = max3(t0, s[q], s[q + 1]);
        t1 = max3(t1, s[q + 2], s[q + 3]);
        t2 = max3(t2, s[q + 4], s[q + 5]);
        t3 = max3(t3, s[q + 6], s[q + 7]);
      }
      t0 = max3(t0, s[kT - 4], s[kT - 3]);
      t1 = max3(t1, s[kT - 2], s[kT - 1]);
      const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3));
      const bool grow = ns == 0 ? top != -INFINITY : (top - mref) * c > kGrow;
      if (ns == 0) {
        mref = top;
      } else if (__any_sync(0xffffffffu, grow)) {
        // O holds the sum up to the previous tile once its product has completed
        if (!(ok = wait(bar(fs.o_done[w]), (ns - 1) & 1u))) break;
        fence_after_sync();
        // between the bases as they are rounded, which is what the weights refer to (from -inf: 0,
        // and O is 0 too)
        const float f = grow ? ex2(__fmul_rn(mref, c) - __fmul_rn(top, c)) : 1.f;
        if (grow) mref = top;
        l2.x *= f;
        l2.y *= f;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          float o[32];
          tmem_ld32(tO + 32 * q, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= f;
          tmem_st32(tO + 32 * q, o);
        }
      }
      const float base = mref == -INFINITY ? 0.f : mref * c;
      const float2 c2 = make_float2(c, c), nb = make_float2(-base, -base);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float pk[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float2 y = fma2(make_float2(s[64 * q + 2 * e], s[64 * q + 2 * e + 1]), c2, nb);
          y.x = ex2(y.x);
          y.y = ex2(y.y);
          l2 = add2(l2, y);
          pk[e] = pack2(y.x, y.y);
        }
        tmem_st32(tS + 32 * q, pk);
      }
      tmem_wait_st();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(fs.p_full[w]));
      ++ns;
    }
    // ---- result ---------------------------------------------------------------------------------
    if (ok && ns > 0) ok = wait(bar(fs.o_done[w]), (ns - 1) & 1u);
    ok = __all_sync(0xffffffffu, ok);
    float l = l2.x + l2.y, base = mref * c;
    uint32_t redo = __ballot_sync(0xffffffffu, ok && ns > 0 && mref != -INFINITY &&
                                                   !(fabsf(base) <= kLarge && l < INFINITY));
    if (__builtin_expect(redo != 0, 0)) {
      fence_after_sync();
      for (; redo; redo &= redo - 1) {
        const int r = __ffs(redo) - 1;
        const float2 x = redo_row<D>(a, m, pt, w, b, h, iw + (warp & 3) * 32 + r, r, tO);
        if (lane == r) base = x.x, l = x.y;
      }
    }
    const size_t row_at = ((size_t)b * a.Hq + h) * a.Tq + i, rows = (size_t)a.B * a.Hq * a.Tq;
    // l is 0 only where nothing is visible; a NaN passes on
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (ok) {
      fence_after_sync();
      __nv_bfloat16* dst = (__nv_bfloat16*)a.o + (((size_t)b * a.Tq + i) * a.Hq + h) * D;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        float o[32];
        if (ns > 0) {
          tmem_ld32(tO + 32 * q, o);
          tmem_wait_ld();
        }
        if (PARTS && i < a.Tq && ns > 0) {           // O as it stands
#pragma unroll
          for (int e = 0; e < 8; ++e)
            reinterpret_cast<float4*>(
                a.part + (((size_t)part * (D / 8) + 4 * q + (e >> 1)) * rows + row_at) * 8)[e & 1] =
                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
        if (!PARTS && i < a.Tq) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            if (ns > 0 && l != 0.f)
              y = make_float4(pack2(o[8 * e] * inv, o[8 * e + 1] * inv),
                              pack2(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                              pack2(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                              pack2(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
            reinterpret_cast<float4*>(dst + 32 * q)[e] = y;
          }
        }
      }
      if (PARTS && i < a.Tq)
        reinterpret_cast<float2*>(a.part + rows * parts * D)[part * rows + row_at] =
            make_float2(base, ns > 0 ? l : 0.f);
      else if (!PARTS && a.lse && i < a.Tq)
        a.lse[row_at] = l == 0.f ? -INFINITY : (base + log2f(l)) * kLn2;
    }
  } else {
    fewer_registers<80>();
    if (warp == 9) {
      // ---- loader -------------------------------------------------------------------------
      const int short_rows = m.len < a.Tk ? m.len : -1;    // rows behind it may hold anything
      bool ok = true, raw = false;
      int done = 0, nraw = 0;
      if (pt.n > 0 && lane == 0) {
        mbar_expect_tx(bar(fs.q_full), 2 * L::TILE);
        for (int w = 0; w < 2; ++w)
          for (int pn = 0; pn < D / 64; ++pn)
            tma_load_4d(sb + L::Q + w * L::TILE + pn * kT * 128, &tm_q, 64 * pn, h, i0 + w * kT, b,
                        bar(fs.q_full));
      }
      for (int x = 0; x < pt.n && ok; ++x) {
        const int s = x & 1, j0 = pt.tile(x) * kT;
        const uint32_t par = (uint32_t)(x >> 1) & 1u;
        ok = wait(bar(fs.k_empty[s]), par ^ 1u);
        if (!ok) break;
        if (lane == 0) {
          mbar_expect_tx(bar(fs.k_full[s]), L::TILE);
          for (int pn = 0; pn < D / 64; ++pn)
            tma_load_4d(sb + L::K + s * L::TILE + pn * kT * 128, &tm_k, 64 * pn, hk, j0, b,
                        bar(fs.k_full[s]));
        }
        done = x + 1;
        ok = wait(bar(fs.v_empty[s]), par ^ 1u);
        if (!ok) break;
        raw = short_rows >= 0 && j0 + kT > short_rows;
        uint64_t* vbar = raw ? bar(fs.v_raw) : bar(fs.v_full[s]);
        if (lane == 0) {
          mbar_expect_tx(vbar, L::TILE);
          for (int pn = 0; pn < D / 64; ++pn)
            tma_load_4d(sb + L::V + s * L::TILE + pn * kT * 128, &tm_v, 64 * pn, hk, j0, b, vbar);
        }
        if (raw) {
          // (a wait that gives up here is drained before the rows are left alone)
          ok = wait(vbar, (uint32_t)nraw & 1u);
          if (!ok) mbar_wait(vbar, (uint32_t)nraw & 1u, kDrain);
          ++nraw;
          zero_rows<D>(sm + L::V + s * L::TILE, kT, max(0, short_rows - j0), lane);
          if (lane == 0) mbar_arrive(bar(fs.v_full[s]));
        }
      }
      // copies in flight land before the CTA leaves, also when some warp gave up
      if (lane == 0 && pt.n > 0) {
        mbar_wait(bar(fs.q_full), 0, kDrain);
        for (int x = max(0, done - 2); x < done; ++x) {
          mbar_wait(bar(fs.k_full[x & 1]), (uint32_t)(x >> 1) & 1u, kDrain);
          if (x + 1 < done || ok) mbar_wait(bar(fs.v_full[x & 1]), (uint32_t)(x >> 1) & 1u, kDrain);
        }
      }
    } else if (warp == 8) {
      // ---- issuing warp -----------------------------------------------------------------------
      constexpr uint32_t id_s = idesc_bf16(kT, kT), id_o = idesc_bf16_mn(kT, D);
      bool ok = pt.n == 0 || wait(bar(fs.q_full), 0);
      uint32_t np[2] = {0, 0};                // P V products issued for each tile
      for (int x = 0; x <= pt.n && ok; ++x) {
        const int s = x & 1, sp = s ^ 1;
        const uint32_t par = (uint32_t)(x >> 1) & 1u, ppar = (uint32_t)((x - 1) >> 1) & 1u;
        const int tl = pt.tile(x), tp = pt.tile(x - 1);
        if (x < pt.n && !(ok = wait(bar(fs.k_full[s]), par))) break;
        if (x > 0 && !(ok = wait(bar(fs.v_full[sp]), ppar))) break;
  #pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (x > 0 && pt.t[w].has(tp)) {
            if (!(ok = wait(bar(fs.p_full[w]), np[w] & 1u))) break;
            fence_after_sync();
  #pragma unroll
            for (int ks = 0; ks < kT / 16; ++ks)
              mma_bf16_ta_w(tb + L::TO + D * w, tb + L::TS + 128 * w + 8 * ks,
                            mnmajor(sb + L::V + sp * L::TILE, kT, ks), id_o, np[w] > 0 || ks > 0);
            mma_commit_w(bar(fs.o_done[w]));
            ++np[w];
          }
          if (x < pt.n && pt.t[w].has(tl)) {
            fence_after_sync();
  #pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              mma_bf16_w(tb + L::TS + 128 * w, kmajor(sb + L::Q + w * L::TILE, kT, ks),
                         kmajor(sb + L::K + s * L::TILE, kT, ks), id_s, ks > 0);
            mma_commit_w(bar(fs.s_full[w]));
          }
        }
        if (!ok) break;
        if (x > 0) mma_commit_w(bar(fs.v_empty[sp]));
        if (x < pt.n) mma_commit_w(bar(fs.k_empty[s]));
      }
      // the products issued here complete before tensor memory is freed
      mma_commit_w(bar(fs.drained));
      mbar_wait(bar(fs.drained), 0, kDrain);
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tb, 512);
}

// The parts' sums joined: 8 channels of a row a thread (they lie [part][channels / 8][row][8], so
// that both sides touch whole lines).
template <int D>
__global__ void __launch_bounds__(256)
attn_forward_join(const AttnArgs a, int parts) {
  constexpr int C8 = D / 8;
  const size_t rows = (size_t)a.B * a.Hq * a.Tq;
  const size_t row = (size_t)blockIdx.x * (256 / C8) + threadIdx.x % (256 / C8);   // (b, h, i)
  const int c8 = threadIdx.x / (256 / C8);
  wait_for_previous();
  if (row >= rows) return;
  const float2* ml = reinterpret_cast<const float2*>(a.part + rows * parts * D);
  float top = -INFINITY;
  for (int p = 0; p < parts; ++p) {
    const float2 s = ml[p * rows + row];
    if (s.y != 0.f) top = fmaxf(top, s.x);
  }
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f), u = o;
  for (int p = 0; p < parts; ++p) {
    const float2 s = ml[p * rows + row];
    if (s.y == 0.f) continue;                     // saw nothing, and may have left nothing
    const float4* src =
        reinterpret_cast<const float4*>(a.part + (((size_t)p * C8 + c8) * rows + row) * 8);
    const float4 x = src[0], y = src[1];
    const float f = ex2(s.x - top);
    l = fmaf(f, s.y, l);
    o.x = fmaf(f, x.x, o.x);
    o.y = fmaf(f, x.y, o.y);
    o.z = fmaf(f, x.z, o.z);
    o.w = fmaf(f, x.w, o.w);
    u.x = fmaf(f, y.x, u.x);
    u.y = fmaf(f, y.y, u.y);
    u.z = fmaf(f, y.z, u.z);
    u.w = fmaf(f, y.w, u.w);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const size_t bh = row / a.Tq, i = row % a.Tq;
  __nv_bfloat16* dst =
      (__nv_bfloat16*)a.o + ((bh / a.Hq * a.Tq + i) * a.Hq + bh % a.Hq) * D + 8 * c8;
  *reinterpret_cast<float4*>(dst) =
      make_float4(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv),
                  pack2(u.x * inv, u.y * inv), pack2(u.z * inv, u.w * inv));
  if (a.lse && c8 == 0) a.lse[row] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
}

// Into how many parts the key tiles of a pair are cut: as many as there are SMs for, of at
// least kLeast tiles each (2 and 4 measured within 5 % of 3 on lengths from 500 to 32768).
int parts_of(const AttnArgs& a) {
  const long ctas = (a.Tq + 2L * kT - 1) / (2 * kT) * a.Hq * a.B;
  long keys = a.Tk;
  if (a.window && keys > (long)a.window + 2 * kT + a.sinks)
    keys = (long)a.window + 2 * kT + a.sinks;
  long p = ctas > 0 ? kSMs / ctas : 1;
  const long most = (keys + kT - 1) / kT / kLeast;
  if (p > most) p = most;
  return p < 1 ? 1 : (int)p;
}

template <int D, bool PARTS>
cudaError_t launch_t(const AttnArgs& a, cudaStream_t st) {
  CUtensorMap mq, mk, mv;
  if (!encode_bthd_bf16(&mq, a.q, a.B, a.Tq, a.Hq, D, 64, kT, true) ||
      !encode_bthd_bf16(&mk, a.k, a.B, a.Tk, a.Hkv, D, 64, kT, true) ||
      !encode_bthd_bf16(&mv, a.v, a.B, a.Tk, a.Hkv, D, 64, kT, true))
    return cudaErrorInvalidValue;
  auto kern = attn_forward_tc<D, PARTS>;
  constexpr int smem = FwdLayout<D>::SMEM;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  const int parts = PARTS ? parts_of(a) : 1;
  const unsigned grid = (unsigned)((a.Tq + 2 * kT - 1) / (2 * kT) * a.Hq * a.B * parts);
  kern<<<grid, kWarpsF * 32, smem, st>>>(mq, mk, mv, a, parts, attn_spin_limit());
  if ((e = cudaGetLastError()) != cudaSuccess || !PARTS) return e;
  const size_t rows = (size_t)a.B * a.Hq * a.Tq;
  return launch_after(attn_forward_join<D>, dim3((unsigned)((rows + 2048 / D - 1) / (2048 / D))),
                      256, 0, st, a, parts);
}

}  // namespace

// Workspace of the parts' sums (0 when no pair is cut).
size_t attn_forward_tc_bytes(const AttnArgs& a) {
  const int parts = parts_of(a);
  return parts == 1 ? 0 : (size_t)parts * a.B * a.Hq * a.Tq * (a.d + 2) * sizeof(float);
}

cudaError_t launch_attn_forward_tc(const AttnArgs& a, cudaStream_t st) {
  if (parts_of(a) > 1) return a.d == 64 ? launch_t<64, true>(a, st) : launch_t<128, true>(a, st);
  return a.d == 64 ? launch_t<64, false>(a, st) : launch_t<128, false>(a, st);
}

}  // namespace gdr
