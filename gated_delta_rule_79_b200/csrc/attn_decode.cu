// Attention of one new token per sequence over a paged key-value cache, and the store of
// new keys and values into the pages (sm_100a).  Mathematics and mask: attn_common.cuh, with
// the query at position lengths[n] - 1.
//
// Bound by HBM: every visible token's key and value are read once for all the query heads
// of their group, 2 d e bytes a token and key head (e bytes an element) against 4 d flops a
// query head.  A sequence's visible tokens (the sinks, then the window) are cut into equal
// parts, each a CTA of four or two warps; a warp streams its own tiles of 16 tokens through a private
// ring of shared-memory stages with 16-byte asynchronous copies, so no barrier stands between
// the loads and the products, and keeps its own running maximum, sum and output.  The warps of
// a CTA join in shared memory, the parts of a sequence in a second small kernel that starts
// while the first one drains.
//
// The lengths are on the device, so the cut is made there: every CTA adds up the batch's visible
// tokens, takes parts of as many tokens as give each CTA that the GPU holds one part (few
// sequences), or a quarter of its share but no less than 1024 (many), and looks up which part is
// its own.  Many parts follow one another on an SM, so there a CTA has two warps, and an SM holds
// twice as many: while one of them starts, which takes it about 3 us, the others read.
//
// bf16 with d = 64 or 128: the products run as m16n8k16 warp matrix instructions, 16 query
// heads as the 16 rows (fewer heads leave rows unused, which costs nothing at this ratio of
// bytes to flops: at 6 TB/s a token of 512 bytes passes an SM every 22 cycles, and its
// products over 16 rows take a few).  Other types run as fp32 dot products, lane = token for
// the scores and lane = channels for the output.
//
// The join reads parts in order, so results do not depend on scheduling.

#include <type_traits>

#include "attn_common.cuh"
#include "once.h"

namespace gdr {
namespace {

using namespace attn;

constexpr int kTile = 16;           // tokens of a warp's tile

// Records a length or page outside the cache (gdr_workspace_status: GDR_ERR_INVALID_ARG).
__device__ __forceinline__ void report(unsigned int* status) {
  if (status) atomicOr(status, 8u);
}

// A sequence's visible tokens, numbered 0 .. count-1: the sinks, then the window.
struct Visible {
  int len, ns, gap, count;
  bool fresh;           // the last one's key and value come with the call
  __device__ __forceinline__ int token(int x) const { return x < ns ? x : x + gap; }
};
__device__ __forceinline__ Visible visible(const PagedArgs& a, int n, bool note) {
  Visible v;
  const int cap = (int)min((long)a.max_pages << a.page_shift, (long)0x7fffffff);
  int len = a.lengths[n];
  v.fresh = a.k_new && len > 0 && len <= cap;
  if (len < 0 || len > cap) {
    if (note) report(a.status);
    len = len < 0 ? 0 : cap;
  }
  v.len = len;
  v.ns = v.gap = 0;
  v.count = len;
  if (a.window && len > a.window) {
    v.ns = min(a.sinks, len - a.window);
    v.gap = len - a.window - v.ns;
    v.count = v.ns + a.window;
  }
  return v;
}
constexpr int kMaxSplit = 256;      // parts of a sequence
constexpr int kLeast = 64;          // tokens of a part, where a sequence is cut at all

// One part: `tokens` visible tokens from part * tokens on (fewer at the end, none in a part behind
// it); `slot` is its place among all parts, -1 for a place behind the last one.
struct Part {
  int n, part, parts, tokens, slot;
};
// The part in place `slot`.  Each warp finds it by itself (no barrier): its lanes count the parts
// of a run of sequences each.  (TIGHT: with the search; its code alone cost the launches that do not
// search 1 %.)
template <bool TIGHT>
__device__ __forceinline__ Part find_part(const PagedArgs& a, int slot) {
  if (a.nparts == 0) return Part{slot, 0, 1, 0x7fffffff, 0};
  auto cut = [&](int n, int at, int parts, int count) {
    // where the join finds the sequence's parts
    if (slot == at && threadIdx.x == 0) a.first[n] = make_int2(at, parts);
    const int tokens = (count + parts - 1) / parts;
    return Part{n, slot - at, parts, max(kLeast, (tokens + kTile - 1) / kTile * kTile), slot};
  };
  if (a.stride) {
    const int n = slot / a.stride, at = n * a.stride;
    const int count = visible(a, n, false).count;
    const int parts = min(kMaxSplit, max(1, (count + kLeast - 1) / kLeast));
    if (slot - at >= parts) return Part{0, 0, 0, 0, -1};
    return cut(n, at, parts, count);
  }
  const int lane = threadIdx.x & 31;
  const int run = (a.N + 31) >> 5;
  const int n0 = min(a.N, lane * run), n1 = min(a.N, n0 + run);
  const int count0 = n0 < n1 ? visible(a, n0, false).count : 0;
  auto count = [&](int n) { return n == n0 ? count0 : visible(a, n, false).count; };
  long long all = count0;
  for (int n = n0 + 1; n < n1; ++n) all += count(n);
#pragma unroll
  for (int f = 16; f; f >>= 1) all += __shfl_xor_sync(0xffffffffu, all, f);
  // no less than all / places (the factor is rounded up), the same in every CTA
  unsigned per =
      max((unsigned)a.least, (unsigned)fminf(__ll2float_ru(all) * a.per_place, 0x1p30f) + 1u);
  auto parts_of = [&](int n) {
    return (int)min((unsigned)kMaxSplit, max(1u, (count(n) + per - 1) / per));
  };
  if (TIGHT && a.tight) {
    // that leaves every sequence a place for a last part, however short; half of them on average
    // stay empty, so halve what lies between it and an even share of all places
    unsigned lo = max((unsigned)a.least, (unsigned)(all / a.nparts));
    unsigned fits = per;
    for (int i = 0; i < 6 && lo < fits; ++i) {
      per = (lo + fits) / 2;
      unsigned sum = 0;
      for (int n = n0; n < n1; ++n) sum += parts_of(n);
      if (__reduce_add_sync(0xffffffffu, sum) <= (unsigned)a.nparts) fits = per;
      else lo = per + 1;
    }
    per = fits;
  }
  const int parts0 = n0 < n1 ? parts_of(n0) : 0;
  int mine = parts0;
  for (int n = n0 + 1; n < n1; ++n) mine += parts_of(n);
  int upto = mine;
#pragma unroll
  for (int f = 1; f < 32; f <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, f);
    if (lane >= f) upto += x;
  }
  const unsigned who = __ballot_sync(0xffffffffu, slot < upto);
  if (who == 0) return Part{0, 0, 0, 0, -1};
  const int src = __ffs(who) - 1;
  int n = n0, c = parts0, at = upto - mine;
  if (lane == src)
    while (slot >= at + c) at += c, c = parts_of(++n);
  n = __shfl_sync(0xffffffffu, n, src);
  at = __shfl_sync(0xffffffffu, at, src);
  c = __shfl_sync(0xffffffffu, c, src);
  return cut(n, at, c, __shfl_sync(0xffffffffu, lane == src ? count(n) : 0, src));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  // takes 16 bytes, or writes zeros when the row is not to be read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               :: "r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
               "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&p);
}

// Where this warp's tile row (a visible token) lies: the row index of the caches, or -1 when
// there is no such token or its page is not one of the pool's; -2 for the new token itself.
struct Rows {
  const PagedArgs& a;
  const Visible& v;
  int n;
  __device__ __forceinline__ long find(int x, int end) const {
    if (x >= end) return -1;
    const int t = v.token(x);
    const int pg = a.table[(size_t)n * a.max_pages + (t >> a.page_shift)];
    if ((unsigned)pg >= (unsigned)a.npages) {
      report(a.status);
      return -1;
    }
    // (also the new token is left out when its page, where it is to be kept, does not exist)
    if (v.fresh && t == v.len - 1) return -2;
    return ((long)pg << a.page_shift) + (t & ((1 << a.page_shift) - 1));
  }
};

// The part that holds the last token stores the new key and value into their page (each key
// head's by the CTA of the group's first 16 heads).  No other CTA touches that row: the
// tokens of a sequence lie in different rows, and sequences do not share their last page.
template <typename T, int D, int W>
__device__ __forceinline__ void store_new(const PagedArgs& a, const Visible& v, int n, int hk) {
  const int t = v.len - 1;
  const int pg = a.table[(size_t)n * a.max_pages + (t >> a.page_shift)];
  if ((unsigned)pg >= (unsigned)a.npages) {
    if (threadIdx.x == 0) report(a.status);
    return;
  }
  const size_t row = ((size_t)pg << a.page_shift) + (t & ((1 << a.page_shift) - 1));
  constexpr int V = 16 / sizeof(T);
  for (int c = threadIdx.x * V; c < 2 * D; c += W * 32 * V) {
    const bool key = c < D;
    const T* src = (const T*)(key ? a.k_new : a.v_new) + ((size_t)n * a.Hkv + hk) * D + c % D;
    T* dst = (T*)(key ? a.kc : a.vc) + (row * a.Hkv + hk) * D + c % D;
    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
  }
}

// Writes one part's result: the output itself when there is only one part, else (o, m, l) of
// the part for the join, with o not yet divided by the sum.
template <typename T>
__device__ __forceinline__ void emit(const PagedArgs& a, const Part& pt, int h, int D, int c,
                                     float o, float m, float l) {
  if (pt.parts == 1) {
    Elem<T>::store((T*)a.o + ((size_t)pt.n * a.Hq + h) * D + c, l != 0.f ? o / l : 0.f);
    return;
  }
  const size_t at = (size_t)pt.slot * a.Hq + h;
  a.part[at * D + c] = o;
  if (c == 0)
    reinterpret_cast<float2*>(a.part + (size_t)a.nparts * a.Hq * D)[at] = make_float2(m, l);
}

template <int D, int W>
struct TcSmem {
  static constexpr int STAGES = 3;
  static constexpr int ROW = D * 2;                       // bytes of a token's key or value
  static constexpr int HALF = kTile * ROW;                // a tile's keys
  static constexpr int PER = STAGES * 2 * HALF;
  static constexpr int RING = W * PER;
  static constexpr int BYTES = RING;                      // the join of the warps reuses it
  static_assert(W * 16 * (D + 4) * 4 + W * 16 * 8 <= RING, "join area");
};

template <int D, int W, bool TIGHT>
__global__ void __launch_bounds__(W * 32)
attn_decode_tc(const PagedArgs a) {
  using S = TcSmem<D, W>;
  using bf16 = __nv_bfloat16;
  extern __shared__ __align__(128) unsigned char sm[];
  let_next_start();
  const int G = a.Hq / a.Hkv, nhb = (G + 15) / 16;
  // the heads of a part run next to each other: their rows are neighbours in the pages
  int x = blockIdx.x;
  const int hb = x % nhb;
  x /= nhb;
  const int hk = x % a.Hkv;
  const Part pt = find_part<TIGHT>(a, x / a.Hkv);
  if (pt.slot < 0) return;
  const int n = pt.n, part = pt.part, parts = pt.parts;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Visible vis = visible(a, n, tid == 0 && part == 0);
  const int h0 = hk * G + hb * 16, nh = min(16, G - hb * 16);
  const int x0 = part * pt.tokens, x1 = x0 + max(0, min(vis.count - x0, pt.tokens));
  if (vis.fresh && hb == 0 && part == parts - 1) store_new<bf16, D, W>(a, vis, n, hk);

  // query fragments, with the scale and log2 e applied to the scores later
  const int g = lane >> 2, t4 = lane & 3;
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int s = 0; s < D / 16; ++s)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int row = g + (u & 1) * 8, col = s * 16 + t4 * 2 + (u >> 1) * 8;
      qf[s][u] = row < nh ? *reinterpret_cast<const uint32_t*>(
                                (const bf16*)a.q + ((size_t)n * a.Hq + h0 + row) * D + col)
                          : 0u;
    }

  // this warp's tiles: warp, warp + 4, ...
  const int ntile = (x1 - x0 + kTile - 1) / kTile;
  const int mine = ntile > warp ? (ntile - warp + W - 1) / W : 0;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sm) + warp * S::PER;
  constexpr int CH = D / 8;                 // 16-byte pieces of a row
  constexpr int RPI = 32 / CH;              // rows a warp instruction copies
  const Rows rows{a, vis, n};
  // lane l < 16 looks up row l of a tile; one tile ahead of the copies
  auto look = [&](int i) -> long {
    return i < mine && lane < kTile ? rows.find(x0 + (warp + i * W) * kTile + lane, x1) : -1;
  };
  auto issue = [&](int i, long mrow) {
    const uint32_t st = ring + (i % S::STAGES) * 2 * S::HALF;
#pragma unroll
    for (int r0 = 0; r0 < kTile; r0 += RPI) {
      const int r = r0 + lane / CH, c = lane % CH;
      const long row = __shfl_sync(0xffffffffu, mrow, r);
      const size_t at = row >= 0 ? ((size_t)row * a.Hkv + hk) * D + c * 8
                                 : ((size_t)n * a.Hkv + hk) * D + c * 8;
      const bool take = row != -1;
      const bf16* kp = (const bf16*)(row == -2 ? a.k_new : a.kc) + (take ? at : 0);
      const bf16* vp = (const bf16*)(row == -2 ? a.v_new : a.vc) + (take ? at : 0);
      const uint32_t dst = st + r * S::ROW + ((c ^ (r & 7)) << 4);
      cp_async16(dst, kp, take);
      cp_async16(dst + S::HALF, vp, take);
    }
  };
  // rows without a token score -inf; the stage's rows are kept as a bit mask of their lanes
  uint32_t live[S::STAGES];
  long ahead = look(0);
#pragma unroll
  for (int i = 0; i < S::STAGES - 1; ++i) {
    live[i] = __ballot_sync(0xffffffffu, ahead != -1);
    if (i < mine) issue(i, ahead);
    cp_commit();
    ahead = look(i + 1);
  }
  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int u = 0; u < 4; ++u) o[i][u] = 0.f;
  float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
  const float c = a.scale * kLog2e;

  // unrolled by the number of stages so that `live` stays in registers
  for (int i0 = 0; i0 < mine; i0 += S::STAGES) {
#pragma unroll
    for (int s = 0; s < S::STAGES; ++s) {
      const int i = i0 + s;
      if (i < mine) {
        const int fill = i + S::STAGES - 1;
        live[(s + S::STAGES - 1) % S::STAGES] = __ballot_sync(0xffffffffu, ahead != -1);
        if (fill < mine) issue(fill, ahead);
        cp_commit();
        ahead = look(fill + 1);
        cp_wait<S::STAGES - 1>();
        __syncwarp();
        const uint32_t st = ring + s * 2 * S::HALF;
        float sc[2][4] = {};
        // scores: B fragments of both 8-token halves from one ldmatrix per 16 channels
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const int r = (lane & 7) + ((lane >> 4) << 3), ch = ks * 2 + ((lane >> 3) & 1);
          uint32_t b[4];
          ldsm4(st + r * S::ROW + ((ch ^ (r & 7)) << 4), b);
          mma_16816(sc[0], qf[ks], b[0], b[1]);
          mma_16816(sc[1], qf[ks], b[2], b[3]);
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const bool on = (live[s] >> (hf * 8 + t4 * 2 + (u & 1))) & 1u;
            sc[hf][u] = on ? sc[hf][u] * c : -INFINITY;
            top[u >> 1] = fmaxf(top[u >> 1], sc[hf][u]);
          }
        float f[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          top[w] = fmaxf(top[w], __shfl_xor_sync(0xffffffffu, top[w], 1));
          top[w] = fmaxf(top[w], __shfl_xor_sync(0xffffffffu, top[w], 2));
          const float now = fmaxf(mx[w], top[w]);
          const float base = now == -INFINITY ? 0.f : now;
          f[w] = exp2f(mx[w] - base);
          mx[w] = now;
          sum[w] *= f[w];
          top[w] = base;
        }
        uint32_t pa[4];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const float p0 = exp2f(sc[hf][2 * w] - top[w]), p1 = exp2f(sc[hf][2 * w + 1] - top[w]);
            sum[w] += p0 + p1;
            pa[hf * 2 + w] = pack_bf16(p0, p1);   // bf16, as the values they weigh
          }
        if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
          for (int e = 0; e < D / 8; ++e) {
            o[e][0] *= f[0];
            o[e][1] *= f[0];
            o[e][2] *= f[1];
            o[e][3] *= f[1];
          }
        }
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
          const int r = lane & 15, ch = e * 2 + (lane >> 4);
          uint32_t b[4];
          ldsm4_t(st + S::HALF + r * S::ROW + ((ch ^ (r & 7)) << 4), b);
          mma_16816(o[2 * e], pa, b[0], b[1]);
          mma_16816(o[2 * e + 1], pa, b[2], b[3]);
        }
        __syncwarp();     // the stage is refilled in the next step
      }
    }
  }
  cp_wait<0>();
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    sum[w] += __shfl_xor_sync(0xffffffffu, sum[w], 1);
    sum[w] += __shfl_xor_sync(0xffffffffu, sum[w], 2);
  }
  __syncthreads();
  float* jo = reinterpret_cast<float*>(sm);                 // [warp][16][D + 4]
  float* jm = jo + W * 16 * (D + 4);                   // [warp][16] m, then l
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int row = g + 8 * w;
#pragma unroll
    for (int e = 0; e < D / 8; ++e) {
      float2 p = make_float2(o[e][2 * w], o[e][2 * w + 1]);
      *reinterpret_cast<float2*>(jo + (warp * 16 + row) * (D + 4) + e * 8 + t4 * 2) = p;
    }
    if (t4 == 0) {
      jm[warp * 16 + row] = mx[w];
      jm[W * 16 + warp * 16 + row] = sum[w];
    }
  }
  __syncthreads();
  for (int e = tid; e < nh * D; e += W * 32) {
    const int row = e / D, ch = e % D;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) m = fmaxf(m, jm[w * 16 + row]);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f, v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = exp2f(jm[w * 16 + row] - base);
      l = fmaf(f, jm[W * 16 + w * 16 + row], l);
      v = fmaf(f, jo[(w * 16 + row) * (D + 4) + ch], v);
    }
    emit<bf16>(a, pt, h0 + row, D, ch, v, m, l);
  }
}

// fp32 arithmetic: a warp's tile is 32 tokens; 8 query heads at a time.
constexpr int kSWarps = 4, kSTile = 32, kSHeads = 8;

template <typename T, int D>
struct SimtSmem {
  float kv[kSWarps][kSTile][D + 4];     // keys, then values; then the warps' outputs
  float q[kSHeads][D];
  float p[kSWarps][kSHeads][kSTile];
  float m[kSWarps][kSHeads], l[kSWarps][kSHeads];
};

template <typename T, int D>
__global__ void __launch_bounds__(kSWarps * 32)
attn_decode_simt(const PagedArgs a) {
  extern __shared__ __align__(128) unsigned char raw[];
  SimtSmem<T, D>& sm = *reinterpret_cast<SimtSmem<T, D>*>(raw);
  let_next_start();
  const int G = a.Hq / a.Hkv, nhb = (G + kSHeads - 1) / kSHeads;
  // the heads of a part run next to each other: their rows are neighbours in the pages
  int x = blockIdx.x;
  const int hb = x % nhb;
  x /= nhb;
  const int hk = x % a.Hkv;
  const Part pt = find_part<true>(a, x / a.Hkv);
  if (pt.slot < 0) return;
  const int n = pt.n, part = pt.part, parts = pt.parts;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Visible vis = visible(a, n, tid == 0 && part == 0);
  const int h0 = hk * G + hb * kSHeads, nh = min(kSHeads, G - hb * kSHeads);
  const int x0 = part * pt.tokens, x1 = x0 + max(0, min(vis.count - x0, pt.tokens));
  if (vis.fresh && hb == 0 && part == parts - 1) store_new<T, D, kSWarps>(a, vis, n, hk);
  for (int e = tid; e < kSHeads * D; e += kSWarps * 32)
    sm.q[e / D][e % D] =
        e / D < nh ? Elem<T>::load((const T*)a.q + ((size_t)n * a.Hq + h0 + e / D) * D + e % D)
                   : 0.f;
  __syncthreads();
  constexpr int CPL = D / 32;            // channels of a lane in the output: lane + 32 e
  float o[kSHeads][CPL] = {}, mx[kSHeads], sum[kSHeads];
#pragma unroll
  for (int h = 0; h < kSHeads; ++h) mx[h] = -INFINITY, sum[h] = 0.f;
  const float c = a.scale * kLog2e;
  const Rows rows{a, vis, n};
  float (*kv)[D + 4] = sm.kv[warp];
  for (int b = x0 + warp * kSTile; b < x1; b += kSWarps * kSTile) {
    const long mrow = rows.find(b + lane, x1);
    auto load = [&](const void* cache, const void* fresh) {
      constexpr int CH = D / 4;
      for (int e = lane; e < kSTile * CH; e += 32) {
        const int r = e / CH, cc = (e % CH) * 4;
        const long row = __shfl_sync(0xffffffffu, mrow, r);
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row >= 0) f = Elem<T>::load4((const T*)cache + ((size_t)row * a.Hkv + hk) * D + cc);
        if (row == -2) f = Elem<T>::load4((const T*)fresh + ((size_t)n * a.Hkv + hk) * D + cc);
        *reinterpret_cast<float4*>(&kv[r][cc]) = f;
      }
    };
    load(a.kc, a.k_new);
    __syncwarp();
    float s[kSHeads] = {};
#pragma unroll 4
    for (int cc = 0; cc < D; cc += 4) {
      const float4 f = *reinterpret_cast<const float4*>(&kv[lane][cc]);
#pragma unroll
      for (int h = 0; h < kSHeads; ++h) {
        const float4 w = *reinterpret_cast<const float4*>(&sm.q[h][cc]);
        s[h] = fmaf(f.x, w.x, fmaf(f.y, w.y, fmaf(f.z, w.z, fmaf(f.w, w.w, s[h]))));
      }
    }
    __syncwarp();
    load(a.vc, a.v_new);
#pragma unroll
    for (int h = 0; h < kSHeads; ++h) {
      s[h] = mrow != -1 ? s[h] * c : -INFINITY;
      float top = s[h];
#pragma unroll
      for (int f = 16; f; f >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, f));
      const float now = fmaxf(mx[h], top), base = now == -INFINITY ? 0.f : now;
      const float f = exp2f(mx[h] - base), p = exp2f(s[h] - base);
      mx[h] = now;
      sum[h] = fmaf(sum[h], f, p);       // this lane's tokens only, until the end
      sm.p[warp][h][lane] = p;
#pragma unroll
      for (int e = 0; e < CPL; ++e) o[h][e] *= f;
    }
    __syncwarp();
#pragma unroll 4
    for (int r = 0; r < kSTile; ++r) {
      float v[CPL];
#pragma unroll
      for (int e = 0; e < CPL; ++e) v[e] = kv[r][lane + 32 * e];
#pragma unroll
      for (int h = 0; h < kSHeads; ++h) {
        const float p = sm.p[warp][h][r];
#pragma unroll
        for (int e = 0; e < CPL; ++e) o[h][e] = fmaf(p, v[e], o[h][e]);
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int h = 0; h < kSHeads; ++h) {
#pragma unroll
    for (int f = 16; f; f >>= 1) sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], f);
#pragma unroll
    for (int e = 0; e < CPL; ++e) kv[h][lane + 32 * e] = o[h][e];
    if (lane == 0) {
      sm.m[warp][h] = mx[h];
      sm.l[warp][h] = sum[h];
    }
  }
  __syncthreads();
  for (int e = tid; e < nh * D; e += kSWarps * 32) {
    const int h = e / D, ch = e % D;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSWarps; ++w) m = fmaxf(m, sm.m[w][h]);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f, v = 0.f;
#pragma unroll
    for (int w = 0; w < kSWarps; ++w) {
      const float f = exp2f(sm.m[w][h] - base);
      l = fmaf(f, sm.l[w][h], l);
      v = fmaf(f, sm.kv[w][h][ch], v);
    }
    emit<T>(a, pt, h0 + h, D, ch, v, m, l);
  }
}

// Joins the parts of each (sequence, query head): four warps take the parts in turn, their
// weights formed by all lanes beforehand, so that the loads of the outputs do not wait for one
// another (a warp alone, a part at a time, took 23 us over 32 parts).

template <typename T, int D>
__global__ void __launch_bounds__(128)
attn_decode_join(const PagedArgs a) {
  __shared__ float wt[kMaxSplit], acc[4][D], red[2][4];
  const int nh = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  wait_for_previous();
  const int2 of = a.first[nh / a.Hq];
  const int parts = of.y;
  if (parts <= 1) return;
  // part s of this head lies s * Hq further on
  const size_t at = (size_t)of.x * a.Hq + nh % a.Hq;
  const float* p = a.part + at * D;
  const float2* ml = reinterpret_cast<const float2*>(a.part + (size_t)a.nparts * a.Hq * D) + at;
  const size_t step = a.Hq;
  constexpr int PT = kMaxSplit / 128;
  float2 x[PT];
  float m = -INFINITY;
#pragma unroll
  for (int e = 0; e < PT; ++e) {
    x[e] = tid + 128 * e < parts ? ml[(tid + 128 * e) * step] : make_float2(-INFINITY, 0.f);
    m = fmaxf(m, x[e].x);
  }
#pragma unroll
  for (int f = 16; f; f >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, f));
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
#pragma unroll
  for (int e = 0; e < PT; ++e) {
    const float f = exp2f(x[e].x - base);
    wt[tid + 128 * e] = f;
    l = fmaf(f, x[e].y, l);
  }
#pragma unroll
  for (int f = 16; f; f >>= 1) l += __shfl_xor_sync(0xffffffffu, l, f);
  if (lane == 0) red[1][warp] = l;
  __syncthreads();
  constexpr int CPL = D / 32;
  float o[CPL] = {};
#pragma unroll 8
  for (int s = warp; s < parts; s += 4) {
    const float f = wt[s];
#pragma unroll
    for (int e = 0; e < CPL; ++e) o[e] = fmaf(f, p[s * step * D + lane + 32 * e], o[e]);
  }
#pragma unroll
  for (int e = 0; e < CPL; ++e) acc[warp][lane + 32 * e] = o[e];
  __syncthreads();
  l = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  const float inv = l != 0.f ? 1.f / l : 0.f;
  if (tid < D)
    Elem<T>::store((T*)a.o + (size_t)nh * D + tid,
                   ((acc[0][tid] + acc[1][tid]) + (acc[2][tid] + acc[3][tid])) * inv);
}

// Token t of sequence n (t < counts[n]) goes to position start[n] + t of its pages: a thread
// for each 16 bytes of keys and values.
__global__ void __launch_bounds__(256)
kv_append_kernel(const AppendArgs a) {
  const size_t total = (size_t)a.N * a.K * a.Hkv * a.pieces;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const size_t row = (size_t)a.Hkv * a.pieces;         // 16-byte pieces of a token
  const int n = (int)(i / (row * a.K));
  const int t = (int)(i / row % a.K);
  const int count = a.counts ? min(a.counts[n], a.K) : a.K;
  if (t >= count) return;
  const long pos = (long)a.start[n] + t;
  if (pos < 0 || pos >= ((long)a.max_pages << a.page_shift)) {
    report(a.status);
    return;
  }
  const int pg = a.table[(size_t)n * a.max_pages + (pos >> a.page_shift)];
  if ((unsigned)pg >= (unsigned)a.npages) {
    report(a.status);
    return;
  }
  const size_t slot = ((size_t)pg << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
  const size_t dst = slot * row + i % row;
  reinterpret_cast<uint4*>(a.kc)[dst] = reinterpret_cast<const uint4*>(a.k)[i];
  reinterpret_cast<uint4*>(a.vc)[dst] = reinterpret_cast<const uint4*>(a.v)[i];
}

template <typename K>
cudaError_t launch_main(K kern, int threads, int smem, const PagedArgs& a, int heads,
                        cudaStream_t st, std::atomic<unsigned long long>& done) {
  cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  const int blocks = (a.Hq / a.Hkv + heads - 1) / heads;
  const unsigned grid = (unsigned)((size_t)(a.nparts ? a.nparts : a.N) * a.Hkv * blocks);
  kern<<<grid, threads, smem, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_t(const PagedArgs& a, cudaStream_t st) {
  cudaError_t e;
  if constexpr (sizeof(T) == 2 && D >= 64) {
    auto go = [&](auto w, auto tight) {
      static std::atomic<unsigned long long> raised{0};
      constexpr int W = decltype(w)::value;
      return launch_main(attn_decode_tc<D, W, decltype(tight)::value>, W * 32, TcSmem<D, W>::BYTES,
                         a, 16, st, raised);
    };
    using std::integral_constant;
    const auto warps = [&](auto w) {
      return a.tight ? go(w, std::true_type{}) : go(w, std::false_type{});
    };
    e = a.four_warps ? warps(integral_constant<int, 4>{}) : warps(integral_constant<int, 2>{});
  } else {
    static std::atomic<unsigned long long> done{0};
    e = launch_main(attn_decode_simt<T, D>, kSWarps * 32, (int)sizeof(SimtSmem<T, D>), a, kSHeads,
                    st, done);
  }
  if (e != cudaSuccess || a.nparts == 0) return e;
  return launch_after(attn_decode_join<T, D>, dim3((unsigned)(a.N * a.Hq)), 128, 0, st, a);
}

// CTAs of `bytes` of shared memory that an SM holds, if a thread takes 128 registers, as it does for
// d = 32 and 64.  For d = 128 it takes up to 209 (bf16, two warps; 168 with four, 149 in fp32), but
// there shared memory leaves room for 4 (2, 3) CTAs only, which still fit.
constexpr int held(int bytes, int threads) {
  const int by_smem = 227 * 1024 / (bytes + 1024), by_regs = 512 / threads;
  return by_smem < by_regs ? by_smem : by_regs;
}

// How the visible tokens are cut (the comment at the top).  The number of places for parts
// follows from the sizes alone; CTAs of places without a part leave after the count.  Few tokens
// need no count: when parts of kLeast have a place each in one round, each sequence has `stride`
// places.  With more than 1024 sequences counting would take too long, and balance is good
// without a cut.  Measured, four warps against two in a single round: 16 sequences of 4096 (8 key
// heads, d = 128) 54 us and 50, 32 with a window of 1024 (2 key heads) 15.0 and 16.7; parts of
// 1024 against 512 in several rounds: 64 sequences of 1000 46 us and 54; the search for the
// shortest parts against places kept for every sequence's last part (8 key heads, d = 128): 37
// sequences of up to 6000 94 us and 112, 32 of up to 8192 105 and 119, 8 of up to 16384 62 and 64
// (64 of up to 8192 with 4 key heads of d = 64: 60 and 58.5).
template <typename T, int D>
void plan_t(PagedArgs& a, long most) {
  constexpr bool tc = sizeof(T) == 2 && D >= 64;
  constexpr int heads = tc ? 16 : kSHeads;
  const long chains = (long)a.Hkv * ((a.Hq / a.Hkv + heads - 1) / heads);
  constexpr int held4 = tc ? held(TcSmem<D, 4>::BYTES, 128) : held(sizeof(SimtSmem<T, D>), 128);
  constexpr int held2 = tc ? held(TcSmem<D, 2>::BYTES, 64) : held4;
  const long round4 = 148L * held4 / chains, round2 = 148L * held2 / chains;
  const bool one = 2L * a.N <= round2;        // (a part of each sequence may be a short one)
  a.four_warps = 3L * a.N <= round4;
  a.least = one ? kLeast : 1024;
  const long places = a.four_warps ? round4 - a.N : one ? round2 - a.N : 4 * round2;
  a.places = places < 1 ? 1 : (int)places;
  a.per_place = 1.0f / (float)a.places * 1.000001f;
  const long each = (most + a.least - 1) / a.least, by_tokens = a.N * each;
  a.stride = a.four_warps && by_tokens <= round4 ? (int)each : 0;
  const long n = a.places + a.N < by_tokens && !a.stride ? a.places + (long)a.N : by_tokens;
  a.nparts = a.N > 1024 || n <= a.N ? 0 : (int)n;
  a.tight = one && a.N <= 64;            // (at most two sequences a lane to add up again)
}

template <typename T>
cudaError_t launch_d(const PagedArgs& a, cudaStream_t st) {
  switch (a.d) {
    case 32: return launch_t<T, 32>(a, st);
    case 64: return launch_t<T, 64>(a, st);
    case 128: return launch_t<T, 128>(a, st);
  }
  return cudaErrorInvalidValue;
}
template <typename T>
void plan_d(PagedArgs& a, long most) {
  if (a.d == 32) plan_t<T, 32>(a, most);
  if (a.d == 64) plan_t<T, 64>(a, most);
  if (a.d == 128) plan_t<T, 128>(a, most);
}

}  // namespace

void attn_decode_plan(PagedArgs& a, long capacity) {
  long most = capacity;
  if (a.window && most > (long)a.window + a.sinks) most = (long)a.window + a.sinks;
  if (a.dtype == GDR_F32) plan_d<float>(a, most);
  else plan_d<__nv_bfloat16>(a, most);
}

cudaError_t launch_attn_decode(const PagedArgs& a, cudaStream_t st) {
  return a.dtype == GDR_F32 ? launch_d<float>(a, st) : launch_d<__nv_bfloat16>(a, st);
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t st) {
  const size_t total = (size_t)a.N * a.K * a.Hkv * a.pieces;
  kv_append_kernel<<<(unsigned)((total + 255) / 256), 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace gdr
