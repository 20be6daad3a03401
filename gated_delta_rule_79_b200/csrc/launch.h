// Internal launcher declarations of libgdr (host side).  The C ABI in gdr.h
// validates arguments and then calls these.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace gdr {

struct PrefillArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* alpha;
  const float* beta;
  const float* s0;      // may be null (zeros)
  void* o;
  float* s_final;       // may be null
  int B, T, H, dk, dv;
  int in_dtype, out_dtype;
  bool kda;
  void* workspace;
  size_t ws_bytes;
  unsigned pro;         // GDR_PROLOGUE_* flags (0: q, k normalised and alpha given)
};

struct DecodeArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* alpha;
  const float* beta;
  float* state;
  void* o;
  int N, H, dk, dv;
  int in_dtype, out_dtype;
  bool kda;
  unsigned pro;         // GDR_PROLOGUE_* flags
};

struct VerifyArgs {
  const void* q;        // [N, K, H, dk]
  const void* k;
  const void* v;        // [N, K, H, dv]
  const float* alpha;   // [N, K, H] or [N, K, H, dk]
  const float* beta;    // [N, K, H]
  float* state;         // [N, H, dv, dk]: read; updated in place when snapshots is null
  float* snapshots;     // [K, N, H, dv, dk] or null
  void* o;              // [N, K, H, dv]
  int N, K, H, dk, dv;
  int in_dtype, out_dtype;
  bool kda;
  unsigned pro;         // GDR_PROLOGUE_* flags
};

struct ChunkMap;   // chunkmap.cuh

// The two-kernel tensor-core prefills (prefill_split.cu, prefill_kda_split.cu): bf16,
// d_k = 128, d_v a multiple of 32.  Chunk images per (head, chunk) in the workspace.
size_t split_prefill_workspace(int B, int T, int H);
size_t kda_split_workspace(int B, int T, int H);
size_t split_chunk_image_bytes();
size_t kda_chunk_image_bytes();
cudaError_t launch_prefill_split(const PrefillArgs& a, const ChunkMap& m, cudaStream_t stream);
cudaError_t launch_prefill_kda_split(const PrefillArgs& a, const ChunkMap& m,
                                     cudaStream_t stream);
// The state carry both two-kernel prefills share, run after the prep kernel has written
// the chunk images; chunk_image_bytes() is the size of one image.  launch_chunk_carry
// (carry_dispatch.cu) picks the chained carry (carry_chain.cu), the per-head carry
// (carry_rows.cu) or the value-sliced one (carry_sliced.cu).
cudaError_t launch_chunk_carry(const PrefillArgs& a, const ChunkMap& m, uint32_t spin_limit,
                               cudaStream_t stream);
cudaError_t launch_carry_rows(const PrefillArgs& a, const ChunkMap& m, uint32_t spin_limit,
                              cudaStream_t stream);
cudaError_t launch_carry_sliced(const PrefillArgs& a, const ChunkMap& m, uint32_t spin_limit,
                                cudaStream_t stream);
cudaError_t launch_carry_chain(const PrefillArgs& a, const ChunkMap& m, uint32_t spin_limit,
                               cudaStream_t stream);
size_t chunk_image_bytes();

// Gradients of a dense prefill (backward.cu).
struct BackwardArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* alpha;
  const float* beta;
  const float* s0;        // may be null (zeros)
  const void* dO;
  const float* ds_final;  // may be null (zeros)
  float* dq_out;
  float* dk_out;
  float* dv_out;
  float* dalpha;
  float* dbeta;
  float* ds0;
  int B, T, H, dk, dv;
  int in_dtype, do_dtype;
  bool kda;
  void* workspace;
};
size_t backward_workspace_bytes(int B, int T, int H, int dk, int dv);
cudaError_t launch_backward(const BackwardArgs& a, cudaStream_t stream);

// ---- linear attention with one decay per head (lin_common.cuh) -------------------------
// One scan over the tokens: the prefill, or one of the three that the gradients are.
struct LinJob {
  const void* q;        // [B, T, H, dk]
  const void* k;        // [B, T, H, dk]
  const void* v;        // [B, T, H, dv]
  void* o;              // [B, T, H, dv]
  const float* s_in;    // [B, H, dv, dk] entering state ([B, H, dk, dv] with s_trans), or null
  float* s_out;         // [B, H, dv, dk], or null
  int rev;              // 1: from the last token to the first
  int e0;               // decay steps between the entering state and the first output (0 or 1)
  int s_trans;
};
constexpr int kLinMaxJobs = 3;
struct LinScan {
  LinJob job[kLinMaxJobs];
  const float* decay;   // [H]
  float* part;          // nseg > 1: [njobs, B, H, nseg] states: in slot p + 1 what segment p left,
                        // then in slot p the state that segment p is entered with
  int part_rows;        // 1: the states in part lie row by row; 0: as lin::part_at says
  unsigned int* status;
  int njobs, B, T, H, dk, dv, dtype;
  int seg_len, nseg;
};
cudaError_t launch_lin_carry(const LinScan& sc, cudaStream_t stream);
cudaError_t launch_lin_tc(const LinScan& sc, cudaStream_t stream);    // bf16, dk and dv >= 64
cudaError_t launch_lin_simt(const LinScan& sc, cudaStream_t stream);

struct LinDecodeArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* decay;
  float* state;
  void* o;
  int N, H, dk, dv, dtype;
};
cudaError_t launch_lin_decode(const LinDecodeArgs& a, cudaStream_t stream);

// ---- softmax attention with a sliding window and sinks (attn_common.cuh) ----------------
struct AttnArgs {
  const void* q;        // [B, Tq, Hq, d]
  const void* k;        // [B, Tk, Hkv, d]
  const void* v;
  const int* lengths;   // [B] or null
  void* o;              // [B, Tq, Hq, d]
  float* lse;           // [B, Hq, Tq] or null (forward only)
  unsigned int* status;
  int B, Tq, Tk, Hq, Hkv, d;
  int window, sinks;    // window 0: none (and then no sinks)
  float scale;
  int dtype;
  float* part;          // workspace of attn_forward_tc_bytes: sums of parts of the keys
};
struct AttnGradArgs {
  AttnArgs f;           // the forward's arguments and results
  const void* dO;
  float* delta;         // [B, Hq, Tq] workspace: do . o of every row
  float* part;          // workspace of attn_backward_.._bytes(f): sums of parts of key tiles
  void* dq;
  void* dk;
  void* dv;
};
cudaError_t launch_attn_forward_simt(const AttnArgs& a, cudaStream_t stream);  // fp32, or d = 32
cudaError_t launch_attn_forward_tc(const AttnArgs& a, cudaStream_t stream);   // bf16, d >= 64
cudaError_t launch_attn_no_keys(const AttnArgs& a, cudaStream_t stream);      // Tk = 0
cudaError_t launch_attn_delta(const AttnGradArgs& a, cudaStream_t stream);
size_t attn_forward_tc_bytes(const AttnArgs& a);
size_t attn_backward_tc_bytes(const AttnArgs& f);
size_t attn_backward_simt_bytes(const AttnArgs& f);
cudaError_t launch_attn_backward_tc(const AttnGradArgs& a, cudaStream_t stream);  // bf16, d >= 64
cudaError_t launch_attn_backward_simt(const AttnGradArgs& a, cudaStream_t stream);

struct PagedArgs {
  const void* q;        // [N, Hq, d]
  const void* k_new;    // [N, Hkv, d] or null
  const void* v_new;
  void* kc;             // [npages, 1 << page_shift, Hkv, d]
  void* vc;
  const int* table;     // [N, max_pages]
  const int* lengths;   // [N]
  void* o;              // [N, Hq, d]
  int2* first;          // [N] a sequence's first part and their number
  float* part;          // [nparts, Hq] x d outputs, then [nparts, Hq] x (max, sum)
  unsigned int* status;
  int N, Hq, Hkv, d, npages, page_shift, max_pages, window, sinks;
  float scale;
  int dtype;
  // parts hold tokens / places of them, but no less than `least`; room for `nparts` (0: uncut)
  int places, least, nparts;
  float per_place;      // 1 / places, rounded up
  int stride;           // places of each sequence, or 0: as the tokens fall
  bool four_warps;      // of a CTA, or two
  bool tight;           // look for the shortest parts that fit `nparts` places
};
void attn_decode_plan(PagedArgs& a, long capacity);   // sets the last seven
cudaError_t launch_attn_decode(const PagedArgs& a, cudaStream_t stream);

struct AppendArgs {
  const void* k;        // [N, K, Hkv, d]
  const void* v;
  void* kc;
  void* vc;
  const int* table;
  const int* start;     // [N]
  const int* counts;    // [N] or null
  unsigned int* status; // may be null
  int N, K, Hkv, pieces, npages, page_shift, max_pages;   // pieces: 16-byte pieces of a row
};
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream);

// Records `msg` as the calling thread's gdr_last_error() text and returns `s`.
int report_error(int s, const char* msg);

// GDR_CHECKS build: the current device's word that failed device-side index checks set
// (checks.cuh), allocated and zeroed on first use; nullptr in the product build (and if
// that allocation failed).
unsigned int* checks_word();

// Measurement aid (timing.cu): records an event on `stream` when timing is on.
// slot -1 marks the start of a prefill call, slot i the end of its i-th kernel.
void timing_mark(cudaStream_t stream, int slot);

// Each returns cudaSuccess or the launch error; messages are set by the caller.
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream);
cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream);
cudaError_t launch_prefill_simt(const PrefillArgs& a, cudaStream_t stream);

}  // namespace gdr
