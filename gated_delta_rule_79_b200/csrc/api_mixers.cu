// C ABI of the linear-attention and softmax-attention mixers (declared in include/gdr.h):
// argument validation, kernel selection and error reporting, as api.cu does for the gated
// delta rule.  Every argument is validated on the host before anything is enqueued.

#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "gdr.h"
#include "launch.h"

namespace gdr {
namespace {

gdr_status fail(gdr_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return (gdr_status)report_error(s, buf);
}
gdr_status ok() { return (gdr_status)report_error(GDR_OK, ""); }
gdr_status done(const char* fn, cudaError_t e) {
  if (e != cudaSuccess)
    return fail(GDR_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return ok();
}

bool head_ok(int d) { return d == 32 || d == 64 || d == 128; }
bool dtype_ok(int t) { return t == GDR_F32 || t == GDR_BF16; }

constexpr size_t kStatusBytes = 256;
constexpr int kSMs = 148;

struct Arg {
  const void* p;
  const char* name;
  bool required;
  int align;
};
template <int N>
gdr_status check_pointers(const char* fn, const Arg (&args)[N]) {
  for (const Arg& a : args) {
    if (a.required && !a.p) return fail(GDR_ERR_INVALID_ARG, "%s: %s is NULL", fn, a.name);
    if (((uintptr_t)a.p & (uintptr_t)(a.align - 1)) != 0)
      return fail(GDR_ERR_INVALID_ARG, "%s: %s is not %d-byte aligned", fn, a.name, a.align);
  }
  return GDR_OK;
}

gdr_status check_workspace(const char* fn, const void* ws, size_t bytes, size_t need) {
  if (!ws || bytes < need)
    return fail(GDR_ERR_INVALID_ARG, "%s: workspace %p of %zu bytes, need %zu", fn, ws, bytes,
                need);
  if (((uintptr_t)ws & 255u) != 0)
    return fail(GDR_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
  return GDR_OK;
}

// ---- linear attention ---------------------------------------------------------------------

bool lin_sizes_ok(int B, int T, int H) {
  return B >= 0 && T >= 0 && H >= 0 && T <= (1 << 28) && (long long)B * H <= (1LL << 22) &&
         (long long)B * T * H <= (1LL << 38);
}

bool lin_tc(int dk, int dv, int dtype) { return dtype == GDR_BF16 && dk >= 64 && dv >= 64; }

// How the tokens are cut.  The tensor-core kernels run one CTA on an SM and stream, so the
// chains (batch, head, scan) are cut until about every SM has one, into no less than 256 tokens;
// every segment but the last reads its keys and values once more.  The CUDA-core kernels are
// bound by arithmetic and want several CTAs on an SM, so there four to an SM, from 64 tokens on.
void lin_cut(long chains, int T, bool tc, int& seg_len, int& nseg) {
  long want = (tc ? kSMs : 4 * kSMs) / (chains > 0 ? chains : 1);
  const long least = tc ? 256 : 64;
  const long most = ((long)T + least - 1) / least;
  if (want > most) want = most;
  if (want < 1) want = 1;
  const long per = (T + want - 1) / want;
  seg_len = (int)((per + 63) / 64 * 64);
  nseg = seg_len > 0 ? (T + seg_len - 1) / seg_len : 1;
  if (nseg < 1) nseg = 1;
}

size_t lin_part_bytes(int B, int T, int H, int dk, int dv, int dtype, int njobs) {
  int seg_len, nseg;
  lin_cut((long)B * H * njobs, T, lin_tc(dk, dv, dtype), seg_len, nseg);
  return nseg > 1 ? (size_t)njobs * B * H * nseg * dk * dv * sizeof(float) : 0;
}

cudaError_t run_scans(LinScan& sc, void* workspace, cudaStream_t st) {
  sc.status = (unsigned int*)workspace;
  sc.part = (float*)((unsigned char*)workspace + kStatusBytes);
  const bool tc = lin_tc(sc.dk, sc.dv, sc.dtype);
  lin_cut((long)sc.B * sc.H * sc.njobs, sc.T, tc, sc.seg_len, sc.nseg);
  sc.part_rows = !tc;
  return tc ? launch_lin_tc(sc, st) : launch_lin_simt(sc, st);
}

gdr_status state_through(const char* fn, const float* in, float* out, size_t bytes,
                         cudaStream_t st) {
  if (!out || (in == out)) return ok();
  return done(fn, in ? cudaMemcpyAsync(out, in, bytes, cudaMemcpyDeviceToDevice, st)
                     : cudaMemsetAsync(out, 0, bytes, st));
}

gdr_status lin_common(const char* fn, int B, int T, int H, int dk, int dv, int dtype) {
  if (B < 0 || T < 0 || H < 0)
    return fail(GDR_ERR_INVALID_ARG, "%s: negative size B=%d T=%d H=%d", fn, B, T, H);
  if (!head_ok(dk) || !head_ok(dv))
    return fail(GDR_ERR_UNSUPPORTED, "%s: d_k=%d d_v=%d (supported: 32, 64, 128)", fn, dk, dv);
  if (!dtype_ok(dtype)) return fail(GDR_ERR_INVALID_ARG, "%s: bad dtype %d", fn, dtype);
  if (!lin_sizes_ok(B, T, H)) return fail(GDR_ERR_INVALID_ARG, "%s: sizes too large", fn);
  return GDR_OK;
}

// ---- softmax attention ----------------------------------------------------------------------

// A window that reaches past every key is none; without one every key is a sink's equal.
void normalise_window(long keys, int& window, int& sinks) {
  if (window <= 0 || window >= keys) window = 0;
  if (window == 0 || sinks < 0) sinks = 0;
  if (sinks > keys) sinks = (int)keys;
}

gdr_status attn_common(const char* fn, int B, int Tq, int Tk, int Hq, int Hkv, int d, int sinks,
                       float scale, int dtype) {
  if (B < 0 || Tq < 0 || Tk < 0 || Hq < 0 || Hkv < 0)
    return fail(GDR_ERR_INVALID_ARG, "%s: negative size B=%d Tq=%d Tk=%d Hq=%d Hkv=%d", fn, B, Tq,
                Tk, Hq, Hkv);
  if (!head_ok(d)) return fail(GDR_ERR_UNSUPPORTED, "%s: d=%d (supported: 32, 64, 128)", fn, d);
  if (!dtype_ok(dtype)) return fail(GDR_ERR_INVALID_ARG, "%s: bad dtype %d", fn, dtype);
  if ((Hkv == 0) != (Hq == 0) || (Hkv > 0 && Hq % Hkv != 0))
    return fail(GDR_ERR_INVALID_ARG, "%s: Hq=%d is not a multiple of Hkv=%d", fn, Hq, Hkv);
  if (sinks < 0) return fail(GDR_ERR_INVALID_ARG, "%s: negative sinks %d", fn, sinks);
  if (!(scale > 0.f) || !isfinite(scale))
    return fail(GDR_ERR_INVALID_ARG, "%s: scale %g is not positive and finite", fn, scale);
  if (Tq > (1 << 28) || Tk > (1 << 28) || (long long)B * Hq > (1LL << 22) ||
      (long long)B * Hq * ((Tq > Tk ? Tq : Tk) / 64 + 1) > (1LL << 30) ||
      (long long)B * Hq * Tq > (1LL << 33))
    return fail(GDR_ERR_INVALID_ARG, "%s: sizes too large", fn);
  return GDR_OK;
}

bool attn_tc(int d, int dtype) { return dtype == GDR_BF16 && d >= 64; }

// Status word, then the sums of cut keys, or (backward) do . o of every row and the sums of cut
// key tiles.  The window is normalised.
size_t attn_delta_bytes(const AttnArgs& a) {
  return ((size_t)a.B * a.Hq * a.Tq * sizeof(float) + 255) / 256 * 256;
}
size_t attn_need(const AttnArgs& a, bool backward) {
  if (a.B == 0 || a.Tq == 0 || a.Tk == 0 || a.Hq == 0) return kStatusBytes;
  const bool tc = attn_tc(a.d, a.dtype);
  if (!backward) return kStatusBytes + (tc ? attn_forward_tc_bytes(a) : 0);
  return kStatusBytes + attn_delta_bytes(a) + (tc ? attn_backward_tc_bytes(a) : attn_backward_simt_bytes(a));
}

int page_shift_of(int page) {
  for (int s = 0; s <= 12; ++s)
    if (page == 1 << s) return s;
  return -1;
}

gdr_status paged_common(const char* fn, int N, int Hq, int Hkv, int d, int npages, int page,
                        int max_pages, int dtype) {
  if (N < 0 || Hq < 0 || Hkv < 0 || npages < 0 || max_pages < 0)
    return fail(GDR_ERR_INVALID_ARG, "%s: negative size N=%d Hq=%d Hkv=%d npages=%d max_pages=%d",
                fn, N, Hq, Hkv, npages, max_pages);
  if (!head_ok(d)) return fail(GDR_ERR_UNSUPPORTED, "%s: d=%d (supported: 32, 64, 128)", fn, d);
  if (!dtype_ok(dtype)) return fail(GDR_ERR_INVALID_ARG, "%s: bad dtype %d", fn, dtype);
  if (page_shift_of(page) < 0)
    return fail(GDR_ERR_UNSUPPORTED, "%s: page=%d (a power of two up to 4096)", fn, page);
  if ((long long)N * Hq > (1LL << 22) || (long long)max_pages * page > (1LL << 30) ||
      (long long)npages * page > (1LL << 40))
    return fail(GDR_ERR_INVALID_ARG, "%s: sizes too large", fn);
  return GDR_OK;
}

// Status word, then (for a batch that is cut) where each sequence's parts lie, and their sums.
size_t first_bytes(int N) { return ((size_t)N * sizeof(int2) + 255) / 256 * 256; }
size_t decode_need(const PagedArgs& a) {
  if (a.nparts == 0) return kStatusBytes;
  return kStatusBytes + first_bytes(a.N) + (size_t)a.nparts * a.Hq * (a.d + 2) * sizeof(float);
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

size_t gdr_lin_workspace_bytes(int B, int T, int H, int dk, int dv, int dtype, int backward) {
  if (!lin_sizes_ok(B, T, H) || !head_ok(dk) || !head_ok(dv) || !dtype_ok(dtype)) return 0;
  size_t part = lin_part_bytes(B, T, H, dk, dv, dtype, 1);
  if (backward) {
    // the scans run together when their head sizes agree, else in two launches
    const size_t all = dk == dv ? lin_part_bytes(B, T, H, dk, dv, dtype, 3)
                                : lin_part_bytes(B, T, H, dk, dv, dtype, 2);
    if (all > part) part = all;
  }
  return kStatusBytes + part;
}

gdr_status lin_prefill(const void* q, const void* k, const void* v, const float* decay,
                       const float* s0, void* o, float* s_final, int B, int T, int H, int dk,
                       int dv, int dtype, void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "lin_prefill";
  gdr_status s = lin_common(fn, B, T, H, dk, dv, dtype);
  if (s != GDR_OK) return s;
  if (B == 0 || H == 0) return ok();
  const bool any = T > 0;
  const Arg args[] = {{q, "q", any, 16}, {k, "k", any, 16}, {v, "v", any, 16},
                      {decay, "decay", any, 4}, {o, "o", any, 16}, {s0, "s0", false, 16},
                      {s_final, "s_final", false, 16}};
  if ((s = check_pointers(fn, args)) != GDR_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  if (T == 0) return state_through(fn, s0, s_final, (size_t)B * H * dk * dv * sizeof(float), st);
  s = check_workspace(fn, workspace, ws_bytes, gdr_lin_workspace_bytes(B, T, H, dk, dv, dtype, 0));
  if (s != GDR_OK) return s;
  LinScan sc{};
  sc.job[0] = LinJob{q, k, v, o, s0, s_final, 0, 1, 0};
  sc.njobs = 1;
  sc.decay = decay;
  sc.B = B, sc.T = T, sc.H = H, sc.dk = dk, sc.dv = dv, sc.dtype = dtype;
  return done(fn, run_scans(sc, workspace, st));
}

gdr_status lin_decode(const void* q, const void* k, const void* v, const float* decay,
                      float* state, void* o, int N, int H, int dk, int dv, int dtype,
                      void* stream) {
  const char* fn = "lin_decode";
  gdr_status s = lin_common(fn, N, 1, H, dk, dv, dtype);
  if (s != GDR_OK) return s;
  if (N == 0 || H == 0) return ok();
  const Arg args[] = {{q, "q", true, 16}, {k, "k", true, 16}, {v, "v", true, 16},
                      {decay, "decay", true, 4}, {state, "state", true, 16}, {o, "o", true, 16}};
  if ((s = check_pointers(fn, args)) != GDR_OK) return s;
  LinDecodeArgs a{q, k, v, decay, state, o, N, H, dk, dv, dtype};
  return done(fn, launch_lin_decode(a, (cudaStream_t)stream));
}

gdr_status lin_backward(const void* q, const void* k, const void* v, const float* decay,
                        const float* s0, const void* dO, const float* ds_final, void* dq,
                        void* dk_out, void* dv_out, float* ds0, int B, int T, int H, int dk,
                        int dv, int dtype, void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "lin_backward";
  gdr_status s = lin_common(fn, B, T, H, dk, dv, dtype);
  if (s != GDR_OK) return s;
  if (B == 0 || H == 0) return ok();
  const bool any = T > 0;
  const Arg args[] = {{q, "q", any, 16}, {k, "k", any, 16}, {v, "v", any, 16},
                      {decay, "decay", any, 4}, {dO, "do", any, 16}, {dq, "dq", any, 16},
                      {dk_out, "dk", any, 16}, {dv_out, "dv", any, 16}, {ds0, "ds0", true, 16},
                      {s0, "s0", false, 16}, {ds_final, "ds_final", false, 16}};
  if ((s = check_pointers(fn, args)) != GDR_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  if (T == 0)
    return state_through(fn, ds_final, ds0, (size_t)B * H * dk * dv * sizeof(float), st);
  s = check_workspace(fn, workspace, ws_bytes, gdr_lin_workspace_bytes(B, T, H, dk, dv, dtype, 1));
  if (s != GDR_OK) return s;
  const LinJob jq{dO, v, k, dq, s0, nullptr, 0, 1, 1};
  const LinJob jk{v, dO, q, dk_out, ds_final, nullptr, 1, 0, 1};
  const LinJob jv{k, q, dO, dv_out, ds_final, ds0, 1, 0, 0};
  LinScan sc{};
  sc.decay = decay;
  sc.B = B, sc.T = T, sc.H = H, sc.dtype = dtype;
  // dq and dk scan with the head sizes exchanged
  sc.dk = dv, sc.dv = dk;
  sc.job[0] = jq;
  sc.job[1] = jk;
  sc.njobs = 2;
  if (dk == dv) {
    sc.job[2] = jv;
    sc.njobs = 3;
  }
  cudaError_t e = run_scans(sc, workspace, st);
  if (e == cudaSuccess && dk != dv) {
    sc.dk = dk, sc.dv = dv;
    sc.job[0] = jv;
    sc.njobs = 1;
    e = run_scans(sc, workspace, st);
  }
  return done(fn, e);
}

size_t gdr_attn_workspace_bytes(int B, int Tq, int Tk, int Hq, int Hkv, int d, int window,
                                int sinks, int dtype, int backward) {
  if (attn_common("gdr_attn_workspace_bytes", B, Tq, Tk, Hq, Hkv, d, sinks, 1.f, dtype) != GDR_OK)
    return 0;
  normalise_window(Tk, window, sinks);
  AttnArgs a{};
  a.B = B, a.Tq = Tq, a.Tk = Tk, a.Hq = Hq, a.Hkv = Hkv, a.d = d;
  a.window = window, a.sinks = sinks, a.dtype = dtype;
  return attn_need(a, backward != 0);
}

gdr_status attn_prefill(const void* q, const void* k, const void* v, const int* lengths, void* o,
                        float* lse, int B, int Tq, int Tk, int Hq, int Hkv, int d, int window,
                        int sinks, float scale, int dtype, void* workspace, size_t ws_bytes,
                        void* stream) {
  const char* fn = "attn_prefill";
  gdr_status s = attn_common(fn, B, Tq, Tk, Hq, Hkv, d, sinks, scale, dtype);
  if (s != GDR_OK) return s;
  if (B == 0 || Hq == 0 || Tq == 0) return ok();
  const Arg args[] = {{q, "q", true, 16}, {k, "k", Tk > 0, 16}, {v, "v", Tk > 0, 16},
                      {o, "o", true, 16}, {lse, "lse", false, 16}, {lengths, "lengths", false, 4}};
  if ((s = check_pointers(fn, args)) != GDR_OK) return s;
  normalise_window(Tk, window, sinks);
  AttnArgs a{q, k, v, lengths, o, lse, (unsigned int*)workspace, B, Tq, Tk, Hq, Hkv, d,
             window, sinks, scale, dtype, (float*)((unsigned char*)workspace + kStatusBytes)};
  if ((s = check_workspace(fn, workspace, ws_bytes, attn_need(a, false))) != GDR_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  if (Tk == 0) return done(fn, launch_attn_no_keys(a, st));
  return done(fn, attn_tc(d, dtype) ? launch_attn_forward_tc(a, st)
                                    : launch_attn_forward_simt(a, st));
}

gdr_status attn_backward(const void* q, const void* k, const void* v, const int* lengths,
                         const void* o, const float* lse, const void* dO, void* dq, void* dk,
                         void* dv, int B, int Tq, int Tk, int Hq, int Hkv, int d, int window,
                         int sinks, float scale, int dtype, void* workspace, size_t ws_bytes,
                         void* stream) {
  const char* fn = "attn_backward";
  gdr_status s = attn_common(fn, B, Tq, Tk, Hq, Hkv, d, sinks, scale, dtype);
  if (s != GDR_OK) return s;
  if (B == 0 || Hq == 0 || (Tq == 0 && Tk == 0)) return ok();
  const bool nq = Tq > 0, nk = Tk > 0;
  const Arg args[] = {{q, "q", nq, 16}, {k, "k", nk, 16}, {v, "v", nk, 16}, {o, "o", nq, 16},
                      {lse, "lse", nq, 16}, {dO, "do", nq, 16}, {dq, "dq", nq, 16},
                      {dk, "dk", nk, 16}, {dv, "dv", nk, 16}, {lengths, "lengths", false, 4}};
  if ((s = check_pointers(fn, args)) != GDR_OK) return s;
  normalise_window(Tk, window, sinks);
  AttnGradArgs a{};
  a.f = AttnArgs{q, k, v, lengths, const_cast<void*>(o), const_cast<float*>(lse),
                 (unsigned int*)workspace, B, Tq, Tk, Hq, Hkv, d, window, sinks, scale, dtype, nullptr};
  a.dO = dO, a.dq = dq, a.dk = dk, a.dv = dv;
  if ((s = check_workspace(fn, workspace, ws_bytes, attn_need(a.f, true))) != GDR_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  const size_t e = dtype == GDR_F32 ? 4 : 2;
  if (Tq == 0 || Tk == 0) {      // nothing sees anything
    cudaError_t r = cudaSuccess;
    if (nq) r = cudaMemsetAsync(dq, 0, (size_t)B * Tq * Hq * d * e, st);
    if (r == cudaSuccess && nk) r = cudaMemsetAsync(dk, 0, (size_t)B * Tk * Hkv * d * e, st);
    if (r == cudaSuccess && nk) r = cudaMemsetAsync(dv, 0, (size_t)B * Tk * Hkv * d * e, st);
    return done(fn, r);
  }
  unsigned char* ws = (unsigned char*)workspace + kStatusBytes;
  a.delta = (float*)ws;
  a.part = (float*)(ws + attn_delta_bytes(a.f));
  cudaError_t r = launch_attn_delta(a, st);
  if (r == cudaSuccess)
    r = attn_tc(d, dtype) ? launch_attn_backward_tc(a, st) : launch_attn_backward_simt(a, st);
  return done(fn, r);
}

size_t gdr_attn_decode_workspace_bytes(int N, int Hq, int Hkv, int d, int page, int max_pages,
                                       int window, int sinks, int dtype) {
  const char* fn = "gdr_attn_decode_workspace_bytes";
  if (paged_common(fn, N, Hq, Hkv, d, 0, page, max_pages, dtype) != GDR_OK) return 0;
  if (N == 0 || Hq == 0 || Hkv == 0 || Hq % Hkv != 0) return kStatusBytes;
  const long cap = (long)max_pages * page;
  normalise_window(cap, window, sinks);
  PagedArgs a{};
  a.N = N, a.Hq = Hq, a.Hkv = Hkv, a.d = d, a.window = window, a.sinks = sinks, a.dtype = dtype;
  attn_decode_plan(a, cap);
  return decode_need(a);
}

gdr_status attn_decode(const void* q, const void* k, const void* v, void* k_cache, void* v_cache,
                       const int* page_table, const int* lengths, void* o, int N, int Hq, int Hkv,
                       int d, int npages, int page, int max_pages, int window, int sinks,
                       float scale, int dtype, void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "attn_decode";
  gdr_status s = paged_common(fn, N, Hq, Hkv, d, npages, page, max_pages, dtype);
  if (s != GDR_OK) return s;
  if ((Hkv == 0) != (Hq == 0) || (Hkv > 0 && Hq % Hkv != 0))
    return fail(GDR_ERR_INVALID_ARG, "%s: Hq=%d is not a multiple of Hkv=%d", fn, Hq, Hkv);
  if (sinks < 0) return fail(GDR_ERR_INVALID_ARG, "%s: negative sinks %d", fn, sinks);
  if (!(scale > 0.f) || !isfinite(scale))
    return fail(GDR_ERR_INVALID_ARG, "%s: scale %g is not positive and finite", fn, scale);
  if ((k == nullptr) != (v == nullptr))
    return fail(GDR_ERR_INVALID_ARG, "%s: k and v are given together or not at all", fn);
  if (N == 0 || Hq == 0) return ok();
  const bool cache = npages > 0;
  const Arg args[] = {{q, "q", true, 16}, {k, "k", false, 16}, {v, "v", false, 16},
                      {k_cache, "k_cache", cache, 16}, {v_cache, "v_cache", cache, 16},
                      {page_table, "page_table", max_pages > 0, 4},
                      {lengths, "lengths", true, 4}, {o, "o", true, 16}};
  if ((s = check_pointers(fn, args)) != GDR_OK) return s;
  const long cap = (long)max_pages * page;
  normalise_window(cap, window, sinks);
  PagedArgs a{q, k, v, k_cache, v_cache, page_table, lengths, o,
              (int2*)((unsigned char*)workspace + kStatusBytes),
              (float*)((unsigned char*)workspace + kStatusBytes + first_bytes(N)),
              (unsigned int*)workspace, N, Hq, Hkv, d, npages, page_shift_of(page), max_pages, window, sinks, scale, dtype,
              0, 0, 0, 0.f, 0, false, false};
  attn_decode_plan(a, cap);
  if ((s = check_workspace(fn, workspace, ws_bytes, decode_need(a))) != GDR_OK) return s;
  return done(fn, launch_attn_decode(a, (cudaStream_t)stream));
}

gdr_status kv_append(const void* k, const void* v, void* k_cache, void* v_cache,
                     const int* page_table, const int* start, const int* counts, int N, int K,
                     int Hkv, int d, int npages, int page, int max_pages, int dtype,
                     void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "kv_append";
  gdr_status s = paged_common(fn, N, Hkv, Hkv, d, npages, page, max_pages, dtype);
  if (s != GDR_OK) return s;
  if (K < 0) return fail(GDR_ERR_INVALID_ARG, "%s: negative K=%d", fn, K);
  if ((long long)N * K * Hkv > (1LL << 34))
    return fail(GDR_ERR_INVALID_ARG, "%s: sizes too large", fn);
  if (N == 0 || K == 0 || Hkv == 0) return ok();
  const bool cache = npages > 0;
  const Arg args[] = {{k, "k", true, 16}, {v, "v", true, 16}, {k_cache, "k_cache", cache, 16},
                      {v_cache, "v_cache", cache, 16},
                      {page_table, "page_table", max_pages > 0, 4}, {start, "start", true, 4},
                      {counts, "counts", false, 4}};
  if ((s = check_pointers(fn, args)) != GDR_OK) return s;
  if (workspace && (s = check_workspace(fn, workspace, ws_bytes, kStatusBytes)) != GDR_OK)
    return s;
  AppendArgs a{k, v, k_cache, v_cache, page_table, start, counts, (unsigned int*)workspace,
               N, K, Hkv, d * (dtype == GDR_F32 ? 4 : 2) / 16, npages, page_shift_of(page),
               max_pages};
  return done(fn, launch_kv_append(a, (cudaStream_t)stream));
}

}  // extern "C"
