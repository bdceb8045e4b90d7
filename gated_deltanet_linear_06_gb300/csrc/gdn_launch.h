// gdn_launch.h -- argument packs and launchers of the libgdn kernels
// (internal to the library; the public surface is include/gdn.h).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

struct DecodeArgs {
  const uint16_t* qkv;     // bf16 [batch][Cc]
  const uint16_t* z;       // bf16 [batch][h_v][128]
  const uint16_t* a;       // bf16 [batch][h_v]
  const uint16_t* b;       // bf16 [batch][h_v]
  const float* A_log;      // [h_v]
  const float* dt_bias;    // [h_v]
  const uint16_t* conv_w;  // bf16 [Cc][4]
  const float* norm_w;     // [128]
  const int32_t* slot;     // nullable [batch]
  float* conv_state;       // [n_slots][3][Cc]
  float* ssm_state;        // [n_slots][h_v][128][128]
  void* out;               // [batch][h_v][128], bf16 or fp32
  int32_t* status;         // nullable device word
  int n_slots, batch, h_k, h_v;
  float l2_eps, rms_eps;
  // multi-token decode (launch_decode_multi): tokens per sequence, the token-major
  // activations above then being [batch][steps][...], and the nullable traces of
  // the states after every token
  int steps;
  float* ssm_trace;        // [batch][steps][h_v][128][128]
  float* conv_trace;       // [batch][steps][3][Cc]
};

struct PrefillArgs {
  const uint16_t* qkv;     // bf16 [T][Cc]
  const uint16_t* z;       // bf16 [T][h_v][128]
  const uint16_t* a;       // bf16 [T][h_v]
  const uint16_t* b;       // bf16 [T][h_v]
  const float* A_log;
  const float* dt_bias;
  const uint16_t* conv_w;  // bf16 [Cc][4]
  const float* norm_w;
  const int32_t* cu_seqlens;  // device [n_seqs + 1]
  float* conv_state;       // [n_seqs][3][Cc]
  float* ssm_state;        // [n_seqs][h_v][128][128]
  uint16_t* out;           // bf16 [T][h_v][128]
  int32_t* status;         // device word (workspace offset 0)
  void* scratch;           // workspace beyond the status word
  size_t scratch_bytes;
  // set by the launcher, inside the scratch area:
  int seg_tokens;          // segment length (sequences up to this long are one segment)
  int* seg_list;           // [count, pad x3][units][8]: the segments of every sequence
  int* multi_list;         // [count, pad x3][slots][4]: sequences longer than one segment
  float* xfer;             // per boundary slot and value head: transfer map, end state, initial state
  int* xzero;              // per boundary slot and value head: 1 where the transfer map is exactly zero
  int* chunk_off;          // [n_seqs + 1]: first chunk record of each sequence (split path; else null)
  int2* chunk_list;        // [max_chunks]: (sequence, first token) of each chunk record, sequence -1 past the end
  uint8_t* rec_kq;         // [max_chunks][h_k] per-chunk key/query tile records
  uint8_t* rec_v;          // [max_chunks][h_v] per-chunk value-head records
  int max_chunks;          // chunk records the workspace holds: total_tokens / 64 + n_seqs
  // the heads one launch of the prep / scan / combine passes covers (a call may
  // run as several head groups): key heads kh0 .. kh0+nkh-1, value heads
  // h0 .. h0+nh-1
  int kh0, nkh, h0, nh;
  int n_seqs, h_k, h_v;
  long long total_tokens;
  float l2_eps, rms_eps;
};

// Slot-to-slot copies of whole states (conv state then SSM state of a slot).
// Pair i copies source slot src_idx[i] (i when src_idx is null) to destination
// slot dst_idx[i] (i when null); with src_conv = src_ssm = null it zeroes the
// destination slot instead.  Slot indices are checked on the device.
struct StateCopyArgs {
  const float* src_conv;
  const float* src_ssm;
  const int32_t* src_idx;
  float* dst_conv;
  float* dst_ssm;
  const int32_t* dst_idx;
  int32_t* status;
  long long conv_floats;  // per slot: (W-1) * Cc
  long long ssm_floats;   // per slot: h_v * d_v * d_k
  int src_slots, dst_slots, n;
};

// Dense projection D = A B^T (bf16 operands, fp32 accumulation, bf16 out):
// A [M][K] and B [N][K] row-major (K contiguous, K % 8 == 0, 16-byte aligned
// bases).  The N output columns are split into runs: columns col0 ..
// col0+ncols-1 go to ptr[row * ld + (col - col0)] (col0, ncols, ld multiples
// of 8, ptr 16-byte aligned).
constexpr int kGemmMaxSegs = 4;
struct GemmOut {
  uint16_t* ptr;
  long long ld;
  int col0, ncols;
};
struct GemmArgs {
  const uint16_t* A;
  const uint16_t* B;
  int M, N, K;
  int nseg;
  GemmOut seg[kGemmMaxSegs];
  int32_t* status;         // nullable device word (bounded waits that give up)
};
cudaError_t launch_gemm(const GemmArgs& g, cudaStream_t stream);

// Host launchers: enqueue on `stream`, return the launch error (or
// cudaSuccess).  Dims are validated by the caller.
cudaError_t launch_decode(const DecodeArgs& p, bool out_f32, cudaStream_t stream);
// p.steps tokens per sequence in one launch (1 <= steps <= kDecodeMaxSteps).
constexpr int kDecodeMaxSteps = 8;
cudaError_t launch_decode_multi(const DecodeArgs& p, bool out_f32, cudaStream_t stream);
// A chain of `steps` single steps in one persistent launch: p's activations
// and output are the chain's step-major buffers ([steps][batch][...]).  The
// state rows stay in registers through the chain; the conv state is read (the
// window before the first step) but not written --
// launch_decode_chain_conv_state writes it afterwards.  The results are
// bit-identical to `steps` launch_decode calls.
cudaError_t launch_decode_chain(const DecodeArgs& p, int steps, bool out_f32, cudaStream_t stream);
cudaError_t launch_decode_chain_conv_state(const DecodeArgs& p, const uint16_t* qkv0, int steps,
                                           cudaStream_t stream);
// n <= 65535 pairs per launch.
cudaError_t launch_state_copy(const StateCopyArgs& p, cudaStream_t stream);
// allow_split = false keeps every sequence in one segment (no transfer maps in
// the scratch); the scratch then needs only prefill_scratch_bytes_unsplit().
cudaError_t launch_prefill(const PrefillArgs& p, cudaStream_t stream, bool allow_split = true);
size_t prefill_scratch_bytes(int n_seqs, int h_k, int h_v, long long total_tokens);
size_t prefill_scratch_bytes_unsplit(int n_seqs);
// The segment length gdn_prefill splits long sequences into on a GPU with `sms`
// SMs, or 0 when it does not split (a whole number of chunks, >= 1024 tokens).
long long prefill_segment_tokens(int n_seqs, int h_v, long long total_tokens, int sms);

// gdn_attn_prep: element strides; null q, k or v leaves that part out.
struct AttnPrepArgs {
  const uint16_t *q, *k, *v;
  long long q_st, q_sh, k_st, k_sh, v_st, v_sh;
  const float *q_w, *k_w;
  const double* inv_freq;
  const int32_t *freq_axis, *pos, *slot;
  uint16_t *q_out, *k_cache, *v_cache;
  int32_t* status;
  long long tokens, cache_rows;
  int h_q, h_kv, d, rot, n_axes, pairs;
  float eps;
};
cudaError_t launch_attn_prep(const AttnPrepArgs& p, cudaStream_t stream);

struct AttnSharedArgs {
  const uint16_t *q, *k_cache, *v_cache, *gate;
  const int32_t *prefix_pages, *tail_pages, *tail_len;
  long long prefix_len, n_pages, gate_st, gate_sh;
  uint16_t* out;
  void* scratch;
  int32_t* status;
  int batch, steps, h_q, h_kv, d, page, tail_width;
  float scale;
};
cudaError_t launch_attn_shared(const AttnSharedArgs& p, cudaStream_t stream);
size_t attn_shared_scratch_bytes(int batch, int steps, int h_q, int h_kv, int d);

struct MoeArgs {
  const uint16_t *x, *w_router, *w_gate_up, *w_down, *s_gate_up, *s_down, *s_gate;
  void* y;
  int32_t* topk_id;
  float* topk_w;
  void* scratch;
  int32_t* status;
  int tokens, hidden, inter, experts, top_k, shared_inter;
  bool renorm, out_f32;
};
cudaError_t launch_moe(const MoeArgs& p, cudaStream_t stream);
size_t moe_scratch_bytes(int tokens, int hidden, int inter, int experts, int top_k, int shared_inter);

// gdn_kv4_store and gdn_kv4_load: rows of k and v into the 4-bit cache and out of it.
// Element strides; a null k or v (k_out or v_out) leaves that part out.
struct Kv4RowsArgs {
  const uint16_t *k, *v;   // of a load: the outputs, to say which there are
  long long k_st, k_sh, v_st, v_sh;
  const int32_t* slot;
  uint8_t* cache;
  void *k_out, *v_out;
  int32_t* status;
  long long tokens, cache_rows;
  int h_kv, d, page_log;   // page: 2^page_log rows
  bool out_f32;
};
cudaError_t launch_kv4_store(const Kv4RowsArgs& p, cudaStream_t stream);
cudaError_t launch_kv4_load(const Kv4RowsArgs& p, cudaStream_t stream);

struct AttnKv4Args {
  const uint16_t *q, *gate;
  const uint8_t* cache;
  const int32_t *table, *len;
  long long n_pages, gate_st, gate_sh;
  uint16_t* out;
  void* scratch;
  int32_t* status;
  int batch, steps, h_q, h_kv, d, page, width;
  float scale;
};
cudaError_t launch_attn_kv4(const AttnKv4Args& p, cudaStream_t stream);
size_t attn_kv4_scratch_bytes(int batch, int steps, int h_q, int h_kv, int d);

// gdn_pages_*: the pool's arrays, lists of sequences (null: 0 .. n - 1), copies of pages.
struct PagePool {
  int n_pages, page, n_seqs, width;
  int32_t *refs, *table, *len;
};
struct PageList {
  const int32_t* seq;
  int n;
};
constexpr int kMaxPageCaches = 128;
struct PageMoves {
  const int32_t *from, *to;        // nullable: pair i is page i
  int32_t* status;
  int n, src_pages, dst_pages;
  int caches;
  int first[kMaxPageCaches + 1];   // a warp's pieces of a page, of the caches before each
  const uint8_t* src[kMaxPageCaches];
  uint8_t* dst[kMaxPageCaches];
  long long bytes[kMaxPageCaches];
};
int page_pieces(size_t page_bytes);
cudaError_t launch_pages_extend(const PagePool& p, const PageList& l, int steps, const int32_t* count, int32_t* slot,
                                void* scratch, int32_t* status, cudaStream_t stream);
cudaError_t launch_pages_trim(const PagePool& p, const PageMoves* caches, const PageList& l, const int32_t* new_len,
                              void* scratch, int32_t* status, cudaStream_t stream);
cudaError_t launch_pages_fork(const PagePool& p, const PageMoves* caches, const int32_t* src, const int32_t* dst, int n,
                              void* scratch, int32_t* status, cudaStream_t stream);
cudaError_t launch_pages_free(const PagePool& p, const PageList& l, void* scratch, int32_t* status, cudaStream_t stream);
cudaError_t launch_pages_compact(const PagePool& p, const PageMoves* caches, int32_t* n_live, void* scratch,
                                 int32_t* status, cudaStream_t stream);
cudaError_t launch_pages_copy(const PageMoves& m, cudaStream_t stream);
size_t pages_scratch_bytes(int n_pages, int n_seqs);

}  // namespace gdn
