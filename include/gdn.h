/*
 * gdn.h -- C ABI of libgdn, the Gated DeltaNet layer on NVIDIA GB300 (sm_103a).
 *
 * The layer.  The source pages name it as the linear-attention layer of
 * hybrid Qwen3.x-style models ("Serving large language models on our own
 * stack", section "Qwen3.5-35B-A3B from a real GGUF"; "Our own inference
 * runtime", section "What it is") and fix its serving properties: a
 * fixed-size recurrent state per sequence, constant regardless of position
 * (llmxabe README, architecture paragraph: ~60 MiB per sequence over 30
 * layers, i.e. 2 MiB fp32 per layer at 32 x 128 x 128), carried across
 * chunked prefill and decode (llmxabe README, the worker diagram:
 * "chunked-prefill scheduler"), and a decode that is bit-identical whether a
 * sequence runs alone or batched with others (llmxabe README, status and
 * "Accuracy is a hard gate" paragraphs).  The pages print no formula; the
 * layer computed here is the gated delta rule, per token t of a sequence:
 *
 *   y_t   = silu(causal depthwise conv_W(x)_t)      over the mixed q|k|v channels
 *   q^    = q / sqrt(|q|^2 + l2_eps) / sqrt(d_k),    k^ = k / sqrt(|k|^2 + l2_eps)
 *   g     = -exp(A_log[h]) * softplus(a_t[h] + dt_bias[h]),   beta = sigmoid(b_t[h])
 *   S_t   = exp(g) S_{t-1} (I - beta k^ k^T) + beta v k^T     (S: d_v x d_k, fp32)
 *   o_t   = S_t q^
 *   out_t = o_t / sqrt(mean(o_t^2) + rms_eps) * norm_w * silu(z_t[h])
 *
 * Value head h reads key head h / (h_v / h_k).  The conv weight w[c][W-1]
 * multiplies the current token and w[c][0] the oldest; there is no conv bias.
 *
 * Conventions for every call:
 *   - The caller owns all memory.  The library never allocates or frees
 *     device memory and never synchronises (gdn_read_device_status is the one
 *     call that waits; gdn_prefill_host from pageable host memory may wait in
 *     the runtime's copies).  The only resources it creates are, once per
 *     device, the side streams and events of gdn_prefill's head groups and of
 *     gdn_prefill_host's copies, and the CUDA graph a gdn_decode_graph handle
 *     owns until it is destroyed.
 *   - Calls are asynchronous on the given stream (a cudaStream_t passed as
 *     void*; NULL = the legacy default stream).  The returned status covers
 *     host-side validation and the launch only.  Device-side checks
 *     (cu_seqlens contents, slot indices, bounded waits) write a code into a
 *     device status word instead of faulting; read it with
 *     gdn_read_device_status.
 *   - On GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED or GDN_ERR_WORKSPACE nothing
 *     was launched and no buffer was touched.  GDN_ERR_CUDA can follow part of
 *     a call's launches; the outputs and states are then undefined.
 *   - All device pointers must be 16-byte aligned.  Tensors are dense and
 *     row-major in the shapes given below.
 *   - A workspace serves one call at a time: calls that may run at once need one each.
 *   - Some calls are several kernels, which may begin while the one before them in
 *     the same call still runs; work enqueued before the call is complete when its
 *     first kernel begins, and the call is when its last one ends.
 *   - Activations (qkv, z, a, b), conv weights and the prefill output are
 *     bf16 (raw uint16 bit patterns).  A_log, dt_bias, norm_w and both
 *     states are fp32.
 *   - The only gdn_dims compiled are d_k = d_v = 128, conv_w = 4, chunk = 64,
 *     h_v / h_k in {1, 2, 4}, h_k <= 64; anything else returns
 *     GDN_ERR_UNSUPPORTED.  The attention and expert calls state their limits.
 *   - No exception crosses this boundary.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gdn_status {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARG = 1,    /* null or misaligned pointer, bad size, inconsistent dims */
  GDN_ERR_UNSUPPORTED = 2,    /* dims outside the compiled fast path, or a limit the call states */
  GDN_ERR_WORKSPACE = 3,      /* workspace missing, misaligned or too small */
  GDN_ERR_CUDA = 4,           /* a CUDA runtime call failed (launch, attribute, copy) */
  GDN_ERR_DEVICE_TIMEOUT = 5, /* device word: a bounded device-side wait gave up */
  GDN_ERR_DEVICE_BOUNDS = 6   /* device word: cu_seqlens, a length or an index out of range */
} gdn_status;

/* Layer dimensions.  d_k / d_v: key / value head size; conv_w: conv width;
 * chunk: prefill chunk length; the epsilons of the two norms. */
typedef struct gdn_dims {
  int h_k;
  int h_v;
  int d_k;
  int d_v;
  int conv_w;
  int chunk;
  float l2_eps;
  float rms_eps;
} gdn_dims;

enum { GDN_DTYPE_BF16 = 0, GDN_DTYPE_F32 = 1 };

/* Library version: major * 10000 + minor * 100 + patch. */
int gdn_version(void);

/* Human-readable name of a status code (static storage, never NULL). */
const char* gdn_status_string(gdn_status status);

/* Bytes of carried state per sequence: the fp32 SSM state
 * [h_v][d_v][d_k] plus the fp32 conv state [conv_w - 1][Cc], with
 * Cc = 2 h_k d_k + h_v d_v.  A snapshot of a sequence is a copy of these
 * bytes (the pages' state "snapshot banks": "Our own inference runtime",
 * section "What it is").  Returns 0 for invalid dims. */
size_t gdn_state_bytes(const gdn_dims* dims);

/* Device workspace gdn_prefill needs for this problem (>= 256 bytes; holds
 * the device status word at offset 0).  Returns 0 for invalid arguments. */
size_t gdn_workspace_bytes(const gdn_dims* dims, int n_seqs, long long total_tokens);

/* The segment length, in tokens, that gdn_prefill on the current device splits
 * the sequences of this problem into: a multiple of the chunk (64), at least
 * 1024, chosen from the token count, the value heads and the SM count; 0 when
 * the call splits nothing (enough sequences to fill the GPU, or too few
 * tokens); -1 for invalid arguments or when no device can be queried.  A
 * chunked-prefill scheduler can use it to align its own boundaries; segments
 * never change results beyond rounding. */
long long gdn_prefill_segment_tokens(const gdn_dims* dims, int n_seqs, long long total_tokens);
/* The same choice for a GPU with `sms` SMs, without touching a device (for
 * schedulers that plan ahead, and for tests); -1 for invalid arguments. */
long long gdn_prefill_segment_tokens_for(const gdn_dims* dims, int n_seqs, long long total_tokens,
                                         int sms);

/*
 * Chunked prefill over cu_seqlens-packed variable-length sequences.
 *
 * Runs the layer over every token of n_seqs sequences packed back to back
 * (no padding), each starting from its carried states, and leaves the
 * states after its last token in place -- so a long prompt can be fed in
 * segments, as a chunked-prefill scheduler does (llmxabe README, worker
 * diagram), and a segment continues exactly where the previous one stopped.
 *
 *   qkv        bf16 [total_tokens][Cc]            channel order q | k | v (input)
 *   z          bf16 [total_tokens][h_v][d_v]      output-gate input (input)
 *   a, b       bf16 [total_tokens][h_v]           decay / write-gate inputs (input)
 *   A_log      fp32 [h_v];  dt_bias fp32 [h_v]    (input)
 *   conv_w     bf16 [Cc][conv_w]                  (input)
 *   norm_w     fp32 [d_v]                         RMSNorm weight, shared by heads (input)
 *   cu_seqlens int32 [n_seqs + 1], DEVICE memory, cu_seqlens[0] = 0,
 *              non-decreasing, cu_seqlens[n_seqs] = total_tokens.  Violations
 *              are caught on the device: the call then writes nothing and sets
 *              GDN_ERR_DEVICE_BOUNDS in the status word.
 *   conv_state fp32 [n_seqs][conv_w - 1][Cc]      in/out: raw inputs of the last
 *              conv_w - 1 tokens, oldest first (zeros = fresh sequence)
 *   ssm_state  fp32 [n_seqs][h_v][d_v][d_k]       in/out (zeros = fresh sequence)
 *   out        bf16 [total_tokens][h_v][d_v]      (output)
 *   workspace  device buffer of >= gdn_workspace_bytes(dims, n_seqs,
 *              total_tokens) bytes, 256-byte aligned; its status word is reset
 *              by the call itself.
 * Empty sequences are allowed and leave their states unchanged.  n_seqs = 0
 * or total_tokens = 0 launches nothing and returns GDN_OK.
 *
 * Streams: when some sequence is split into segments (few sequences, so one
 * CTA per (sequence, value head) would leave the GPU short) and h_k is a
 * multiple of 4, the call runs as 4 groups of key heads: the first on `stream`,
 * the others on side streams of the library that wait for `stream` through an
 * event and that `stream` waits for again before the call's last kernel.  Work
 * enqueued on `stream` afterwards therefore sees the call complete, as with a
 * single-stream call; it also works under stream capture.  Concurrent calls
 * on one device from several host threads share the side streams (and are
 * ordered on them).
 */
gdn_status gdn_prefill(const gdn_dims* dims, const void* qkv, const void* z,
                       const void* a, const void* b, const float* A_log,
                       const float* dt_bias, const void* conv_w,
                       const float* norm_w, const int32_t* cu_seqlens,
                       int n_seqs, long long total_tokens, float* conv_state,
                       float* ssm_state, void* out, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * One decode step for a batch of sequences, one token each.
 *
 * Per sequence this is the same arithmetic in the same order whatever the
 * batch size or the batch's other members: a sequence decodes bit-identically
 * alone or batched (llmxabe README, "Accuracy is a hard gate" paragraph).
 *
 *   qkv  bf16 [batch][Cc];  z bf16 [batch][h_v][d_v];  a, b bf16 [batch][h_v]
 *   A_log, dt_bias, conv_w, norm_w   as for gdn_prefill
 *   slot       NULL: batch entry i uses state i of the arrays below.
 *              Else int32 [batch] DEVICE memory: entry i uses state slot[i],
 *              0 <= slot[i] < n_slots, all distinct.  An out-of-range entry
 *              is skipped on the device (its out row is left untouched) and
 *              GDN_ERR_DEVICE_BOUNDS is written to *device_status if given.
 *   n_slots    number of states in the arrays (>= batch when slot is NULL).
 *   conv_state fp32 [n_slots][conv_w - 1][Cc]   in/out
 *   ssm_state  fp32 [n_slots][h_v][d_v][d_k]    in/out
 *   out        [batch][h_v][d_v], bf16 or fp32 per out_dtype (output)
 *   device_status  NULL or a device int32 word that device checks write into
 *              (never cleared by this call).
 * batch = 0 launches nothing and returns GDN_OK.
 */
gdn_status gdn_decode_step(const gdn_dims* dims, const void* qkv, const void* z,
                           const void* a, const void* b, const float* A_log,
                           const float* dt_bias, const void* conv_w,
                           const float* norm_w, const int32_t* slot,
                           int n_slots, int batch, float* conv_state,
                           float* ssm_state, void* out, int out_dtype,
                           int32_t* device_status, void* stream);

/*
 * gdn_decode_step with the step's activations and output in HOST memory, for a
 * serving loop that keeps each step's tokens on the host (llmxabe README,
 * worker diagram: the worker owns the host side of every step).  The step
 * runs on `stream` as gdn_decode_step does (same bits).  When all five host
 * buffers are page-locked memory the device can address, its kernel reads the
 * inputs and writes the output in place over the host link (no copies);
 * otherwise qkv, z, a and b are first copied into the workspace and the output
 * is copied to `out` after the step, on `stream`.
 *
 *   qkv, z, a, b   HOST, layouts as for gdn_decode_step; page-locked memory
 *                  (cudaHostAlloc, torch pin_memory) is used in place,
 *                  pageable memory still works (the copies then block the
 *                  calling thread)
 *   out            HOST [batch][h_v][d_v], bf16 or fp32 per out_dtype (output;
 *                  written once the stream reaches the end of the call)
 *   A_log, dt_bias, conv_w, norm_w, slot, conv_state, ssm_state, device_status
 *                  DEVICE, as for gdn_decode_step
 *   workspace      DEVICE, 256-byte aligned, >= the bytes below (staging for
 *                  the step's inputs and output when they are copied; not
 *                  touched by other calls)
 * The host buffers are read and written when the stream executes the call:
 * leave the inputs unchanged and do not read `out` until the stream has passed
 * it (as with any asynchronous copy).  Every argument is checked before
 * anything is enqueued.  batch = 0 does nothing and returns GDN_OK.
 */
size_t gdn_decode_step_host_workspace_bytes(const gdn_dims* dims, int batch, int out_dtype);
gdn_status gdn_decode_step_host(const gdn_dims* dims, const void* qkv, const void* z,
                                const void* a, const void* b, const float* A_log,
                                const float* dt_bias, const void* conv_w,
                                const float* norm_w, const int32_t* slot, int n_slots,
                                int batch, float* conv_state, float* ssm_state, void* out,
                                int out_dtype, int32_t* device_status, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * gdn_prefill with the activations in HOST memory: the call copies the inputs
 * in and the output out itself, overlapping the host link with the compute.
 *
 * The packed tokens are cut into segments of seg_tokens (0: 5120) tokens, fed
 * as a chunked-prefill scheduler would (llmxabe README, worker diagram): each
 * segment is one gdn_prefill call whose sequences continue from the states the
 * previous segment left.  Two library copy streams move segment i+1's inputs
 * host->device and segment i-1's output device->host while segment i computes.
 * The result equals those gdn_prefill calls made one after another (a segment
 * boundary inside a sequence changes rounding only, as any chunked prefill).
 *
 *   qkv, z, a, b   HOST bf16, layouts as for gdn_prefill; pinned (page-locked)
 *                  memory lets the copies overlap, pageable memory still works
 *   A_log, dt_bias, conv_w, norm_w   DEVICE, as for gdn_prefill
 *   cu_seqlens     HOST int32 [n_seqs + 1], read during the call (checked on
 *                  the host: 0 first, non-decreasing, total_tokens last)
 *   conv_state, ssm_state            DEVICE, in/out, as for gdn_prefill
 *   out            HOST bf16 [total_tokens][h_v][d_v] (output)
 *   seg_tokens     0 or >= 64
 *   workspace      DEVICE, 256-byte aligned, >= gdn_prefill_host_workspace_bytes();
 *                  the int32 at offset 0 holds the first nonzero device status of
 *                  any segment (read it with gdn_read_device_status)
 * Everything is ordered after the caller's earlier work on `stream`, and work
 * enqueued on `stream` afterwards sees the output in host memory.  Not for
 * stream capture.  Concurrent calls on one device share the copy streams.
 */
size_t gdn_prefill_host_workspace_bytes(const gdn_dims* dims, int n_seqs, long long total_tokens,
                                        int seg_tokens);
/*
 * The segments gdn_prefill_host cuts a batch into (host only, no device use):
 * returns their count, or -1 for invalid arguments (cu_seqlens as for
 * gdn_prefill_host, seg_tokens 0 or >= 64), and writes the first max_segs of
 * them to seg_info as {first token, end token, first sequence, sequence
 * count}.  Segment i covers tokens [i * seg, min((i + 1) * seg, total)) and the
 * sequences from the one holding its first token to the one holding its last;
 * an empty sequence at a segment boundary belongs to no segment (its states
 * stay as they are).
 */
long long gdn_prefill_host_segments(const int32_t* cu_seqlens, int n_seqs, long long total_tokens,
                                    int seg_tokens, long long* seg_info, long long max_segs);
gdn_status gdn_prefill_host(const gdn_dims* dims, const void* qkv, const void* z, const void* a,
                            const void* b, const float* A_log, const float* dt_bias,
                            const void* conv_w, const float* norm_w, const int32_t* cu_seqlens,
                            int n_seqs, long long total_tokens, float* conv_state,
                            float* ssm_state, void* out, int seg_tokens, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * Copy whole sequence states between slots of caller-owned state pools:
 * snapshot a prefix's state into a bank and restore it later, or fork one
 * sequence's state into several ("xwen" README, batch mode: the shared prefix
 * is prefilled once and restored for every item; "Our own inference runtime",
 * section "What it is": state "snapshot banks").  The copy is exact, so
 * decoding or prefilling from a restored state gives, bit for bit, what the
 * uninterrupted run gives.
 *
 *   src_conv_state, src_ssm_state  fp32 [src_slots][W-1][Cc], [src_slots][h_v][d_v][d_k]
 *   dst_conv_state, dst_ssm_state  fp32 [dst_slots][...] the same per-slot layout (output)
 *   src_slot, dst_slot  NULL (pair i uses slot i; the pool then needs >= n slots)
 *              or int32 [n] DEVICE arrays of slot indices.  A pair whose index is
 *              out of range is skipped on the device and GDN_ERR_DEVICE_BOUNDS is
 *              written to *device_status if given.
 *   n          pairs, 0 .. 65535 (0 launches nothing)
 * The source and destination slots of one call must not overlap, and no
 * destination slot may appear twice (the copies run concurrently).  Any dims
 * gdn_decode_step accepts; other dims return the same status it does.
 */
gdn_status gdn_state_copy(const gdn_dims* dims, const float* src_conv_state,
                          const float* src_ssm_state, int src_slots, const int32_t* src_slot,
                          float* dst_conv_state, float* dst_ssm_state, int dst_slots,
                          const int32_t* dst_slot, int n, int32_t* device_status, void* stream);

/*
 * Zero the conv and SSM states of n slots of a state pool: the start of a new
 * sequence in a reused slot.  Arguments as for gdn_state_copy's destination.
 */
gdn_status gdn_state_reset(const gdn_dims* dims, float* conv_state, float* ssm_state, int n_slots,
                           const int32_t* slot, int n, int32_t* device_status, void* stream);

/*
 * A CUDA graph of `steps` successive gdn_decode_step calls, for small batches
 * whose steps are launch-bound (three sequences decode a step in a few
 * microseconds of HBM time).  The buffers are bound when the graph is
 * created; the caller refills them between launches.
 *
 *   qkv  bf16 [steps][batch][Cc];  z bf16 [steps][batch][h_v][d_v];
 *   a, b bf16 [steps][batch][h_v]     step t's tokens at [t]
 *   out        [steps][batch][h_v][d_v], bf16 or fp32 per out_dtype
 *   the rest   as for gdn_decode_step (the states advance by `steps` tokens
 *              per launch)
 *   steps 1 .. 2^20, batch >= 1
 *   *graph     receives the handle (NULL on failure)
 * gdn_decode_graph_launch enqueues one run of all the steps on `stream`;
 * results are bit-identical to the same gdn_decode_step calls made one by
 * one.  gdn_decode_graph_destroy frees the handle (NULL is a no-op); the
 * caller must not destroy a graph with a launch still in flight.
 */
typedef struct gdn_decode_graph gdn_decode_graph;

gdn_status gdn_decode_graph_create(const gdn_dims* dims, int steps, const void* qkv, const void* z,
                                   const void* a, const void* b, const float* A_log,
                                   const float* dt_bias, const void* conv_w, const float* norm_w,
                                   const int32_t* slot, int n_slots, int batch, float* conv_state,
                                   float* ssm_state, void* out, int out_dtype,
                                   int32_t* device_status, gdn_decode_graph** graph);
gdn_status gdn_decode_graph_launch(gdn_decode_graph* graph, void* stream);
void gdn_decode_graph_destroy(gdn_decode_graph* graph);

/*
 * Self-test of the device-side failure path.  Launches one CTA whose threads
 * wait, with the kernels' bounded wait and a budget of budget_cycles clock
 * cycles (1 .. 2^31; about 2 GHz), on a shared-memory barrier that nothing
 * completes.  The wait gives up, GDN_ERR_DEVICE_TIMEOUT is written to
 * *device_status (a device int32, left alone if it already holds a code) and
 * the kernel exits; the context stays usable.  The status returned covers the
 * launch only.
 */
gdn_status gdn_selftest_wait_timeout(int32_t* device_status, long long budget_cycles, void* stream);

/* Most tokens per sequence one gdn_decode_multi call takes. */
#define GDN_DECODE_MAX_STEPS 8

/*
 * `steps` decode steps per sequence in one call: multi-token decode, or the
 * verification pass of speculative decoding (the draft tokens of every
 * sequence at once).  The result is bit-identical to `steps` successive
 * gdn_decode_step calls on the same tokens -- every step repeats that call's
 * arithmetic in its order -- while each state is read and written once per
 * call instead of once per token.
 *
 *   qkv  bf16 [batch][steps][Cc];  z bf16 [batch][steps][h_v][d_v];
 *   a, b bf16 [batch][steps][h_v]  (token t of sequence i at [i][t])
 *   A_log, dt_bias, conv_w, norm_w, slot, n_slots, conv_state, ssm_state,
 *   device_status   as for gdn_decode_step; the states end after the last token
 *   steps      1 .. GDN_DECODE_MAX_STEPS
 *   out        [batch][steps][h_v][d_v], bf16 or fp32 per out_dtype (output)
 *   ssm_trace  NULL, or fp32 [batch][steps][h_v][d_v][d_k]: the SSM state after
 *              each token (for rolling back to the last accepted draft token);
 *              it costs one more state write per token
 *   conv_trace NULL, or fp32 [batch][steps][conv_w - 1][Cc]: the conv state
 *              after each token
 * batch = 0 launches nothing and returns GDN_OK.
 */
gdn_status gdn_decode_multi(const gdn_dims* dims, const void* qkv, const void* z,
                            const void* a, const void* b, const float* A_log,
                            const float* dt_bias, const void* conv_w, const float* norm_w,
                            const int32_t* slot, int n_slots, int batch, int steps,
                            float* conv_state, float* ssm_state, void* out, int out_dtype,
                            float* ssm_trace, float* conv_trace, int32_t* device_status,
                            void* stream);

/*
 * Prefill for callers that cannot allocate device memory.
 *
 * The source pages have no counterpart to this call: it exists for callers
 * that cannot hand the library a device workspace at the point where they run
 * the layer -- for instance a step recorded under a strict memory budget, an
 * allocator that forbids new device allocations after start-up, or a host
 * framework that gives the layer no allocation hook.  It computes the same
 * prefill as gdn_prefill (same arguments, layouts and outputs) and allocates
 * nothing: its scratch -- the device status word and the segment list --
 * lives in one fixed device array of GDN_NOALLOC_SCRATCH_BYTES bytes inside
 * the library, which every GPU that loads the library holds until the process
 * exits.
 *
 * Limits and behaviour:
 *   - n_seqs above GDN_NOALLOC_MAX_SEQS returns GDN_ERR_UNSUPPORTED without
 *     launching (the fixed array holds no more).
 *   - Sequences are never split into parallel segments (that needs transfer
 *     maps far larger than the fixed array), so a batch of few long sequences
 *     runs slower than through gdn_prefill; the results agree within the
 *     prefill tolerance.
 *   - The first call in a CUDA context looks up the array's device address
 *     (once per context, with that context's device current) and caches it
 *     under the context's id, so a context rebuilt after cudaDeviceReset looks
 *     it up again; make that first call before any stream capture.
 *   - All calls share the one array, which keeps the previous call's
 *     contents; each call clears the status word itself.  Calls whose work
 *     overlaps on the GPU (other streams, other host threads, concurrent
 *     graph launches) race on the array and must be serialised by the caller.
 *   - device_status: NULL, or a device int32 word that receives a copy of the
 *     call's status word (GDN_OK or the first device-side error) in stream
 *     order, for gdn_read_device_status.  With NULL the device-side errors of
 *     the call are lost: a rejected cu_seqlens (GDN_ERR_DEVICE_BOUNDS, nothing
 *     written, so out and the states keep their old contents) or a bounded
 *     wait that gave up (GDN_ERR_DEVICE_TIMEOUT) goes only to the library's
 *     internal word, which the next call clears.
 */
#define GDN_NOALLOC_MAX_SEQS 32768
#define GDN_NOALLOC_SCRATCH_BYTES 1049344 /* status word + segment list for GDN_NOALLOC_MAX_SEQS */

gdn_status gdn_prefill_noalloc(const gdn_dims* dims, const void* qkv, const void* z,
                               const void* a, const void* b, const float* A_log,
                               const float* dt_bias, const void* conv_w,
                               const float* norm_w, const int32_t* cu_seqlens,
                               int n_seqs, long long total_tokens, float* conv_state,
                               float* ssm_state, void* out, int32_t* device_status,
                               void* stream);

/*
 * The dense projections around the layer.  In the hybrid models the pages
 * run, every Gated DeltaNet layer sits between an input projection of the
 * hidden state and an output projection back to it ("Serving large language
 * models on our own stack", section "Qwen3.5-35B-A3B from a real GGUF";
 * llmxabe README, architecture paragraph: three Gated DeltaNet layers per
 * gated-attention layer).  Both are y = x w^T on the tensor cores, with bf16
 * operands, fp32 accumulation and the result rounded to bf16 (nearest even).
 * Weights are in the output-features-by-input-features layout.
 *
 * gdn_in_proj writes its output columns straight into the layer's input
 * buffers, in the layouts gdn_prefill and gdn_decode_step read, so nothing is
 * copied between the projection and the layer:
 *   x      bf16 [tokens][hidden]                    (input)
 *   w_in   bf16 [Cc + h_v d_v + 2 h_v][hidden]      rows in the order: the Cc
 *          mixed q|k|v conv channels, z (value head major), a (h_v), b (h_v)
 *   qkv    bf16 [tokens][Cc];  z bf16 [tokens][h_v][d_v];
 *   a, b   bf16 [tokens][h_v]                       (outputs)
 *
 * gdn_out_proj maps the layer's output to the hidden size:
 *   o      bf16 [tokens][h_v][d_v]                  (the gdn_prefill / bf16 decode output)
 *   w_out  bf16 [hidden][h_v d_v]
 *   y      bf16 [tokens][hidden]                    (output)
 *
 * hidden: a multiple of 64, at most 65536 (else GDN_ERR_UNSUPPORTED); h_v a
 * multiple of 8; tokens 0 .. 2^31 - 1 (0 launches nothing); dims as for
 * gdn_prefill.  device_status: NULL or a device int32 word that a bounded
 * wait that gave up writes GDN_ERR_DEVICE_TIMEOUT into.  The kernel keeps one
 * CTA per SM resident for the call and uses all of its tensor memory.
 */
gdn_status gdn_in_proj(const gdn_dims* dims, int hidden, long long tokens, const void* x,
                       const void* w_in, void* qkv, void* z, void* a, void* b,
                       int32_t* device_status, void* stream);
gdn_status gdn_out_proj(const gdn_dims* dims, int hidden, long long tokens, const void* o,
                        const void* w_out, void* y, int32_t* device_status, void* stream);

/*
 * The other two blocks of a hybrid model's decode step.  In the models the
 * pages run, every fourth layer is a gated-attention layer with a growing KV
 * cache in place of the recurrent state, and every layer is followed by a
 * mixture-of-experts block (llmxabe README, architecture paragraph).  Three
 * calls cover what lies between their dense projections:
 *   gdn_attn_prep            q and k norms, rotary positions, cache write
 *   gdn_attn_decode_shared   attention of a batch that shares a long prefix
 *   gdn_moe_step             a whole mixture-of-experts layer, few tokens
 *
 * Attention dimensions.  h_q query heads read h_kv key/value heads (query head
 * h reads h / (h_q / h_kv)); d: head size, 64, 128 or 256; rot: rotated
 * dimensions, the first rot of d, a multiple of 16, 0 for none; n_axes: position
 * axes (1 .. GDN_ATTN_MAX_AXES; time, height and width of pictures and video
 * are three); rope_pairs: 0 turns dimension i with i + rot/2, 1 turns 2i with
 * 2i + 1; norm_eps: of the RMS norms; scale: of the scores, 0 for 1/sqrt(d).
 *
 * Cache.  k_cache and v_cache are bf16 [pages][page][h_kv][d], dense: row
 * r = page_index * page + offset holds one token.
 */
typedef struct gdn_attn_dims {
  int h_q;
  int h_kv;
  int d;
  int rot;
  int n_axes;
  int rope_pairs;
  float norm_eps;
  float scale;
} gdn_attn_dims;

#define GDN_ATTN_MAX_AXES 4
#define GDN_ATTN_MAX_STEPS 8    /* most tokens per sequence of gdn_attn_decode_shared */
#define GDN_ATTN_MAX_BATCH 1024 /* most sequences of gdn_attn_decode_shared */
#define GDN_ATTN_MAX_ROWS 128   /* most steps * (h_q / h_kv) */

/*
 * q and k norms, rotary positions and the cache write, in one pass over a
 * token's heads.  Per head x of q and k:
 *   y   = x / sqrt(mean(x^2) + norm_eps) * w
 *   phi = pos[axis(i)][t] * inv_freq[i],  i = 0 .. rot/2 - 1
 *   (y_a, y_b) <- (y_a cos phi - y_b sin phi, y_b cos phi + y_a sin phi)
 * all in fp32, rounded once to bf16.  The angle is reduced to a fraction of a
 * turn in 64-bit fixed point, so far positions lose nothing.
 *
 *   q, k, v    bf16, element strides (token, head) each, both multiples of 8, the
 *              d elements of a head contiguous: dense arrays or views of a
 *              projection's output.  A null q, k or v leaves that part out.
 *   q_norm_w, k_norm_w  fp32 [d], or null for no norm
 *   inv_freq   fp64 [rot / 2], radians per position (null when rot is 0)
 *   freq_axis  int32 [rot / 2], the axis of each frequency; null when n_axes is 1
 *   pos        int32 [n_axes][tokens] (null when rot is 0)
 *   slot       int32 [tokens]: the cache row of each token; negative: not stored.
 *              Null: token t goes to row t.
 *   cache_rows rows of the caches (pages * page); a slot or an axis outside its
 *              range sets GDN_ERR_DEVICE_BOUNDS and the row is not stored (an
 *              axis out of range reads as axis 0)
 *   q_out      bf16 [tokens][h_q][d]; it may be q itself when q is dense
 *   k_cache, v_cache  bf16 [cache_rows][h_kv][d]
 * Slots that are not negative have to differ: of two tokens with the same slot, each
 * 16 bytes of the row in either cache may be the one's or the other's.
 */
gdn_status gdn_attn_prep(const gdn_attn_dims* dims, long long tokens, const void* q,
                         long long q_token_stride, long long q_head_stride, const void* k,
                         long long k_token_stride, long long k_head_stride, const void* v,
                         long long v_token_stride, long long v_head_stride,
                         const float* q_norm_w, const float* k_norm_w, const double* inv_freq,
                         const int32_t* freq_axis, const int32_t* pos, const int32_t* slot,
                         long long cache_rows, void* q_out, void* k_cache, void* v_cache,
                         int32_t* device_status, void* stream);

/*
 * Attention of a batch of sequences that share one prefix.  Sequence b has
 * `steps` query tokens (1 in plain decode, more when drafted tokens are
 * verified) and attends to the prefix's prefix_len tokens and then to its own
 * tail of tail_len[b] tokens, the last `steps` of which are the query tokens
 * themselves: query i sees the tail's tokens 0 .. tail_len[b] - steps + i.
 *   out = softmax(scale q [K_prefix; K_tail]^T) [V_prefix; V_tail] * sigmoid(gate)
 * The prefix is read once for the whole batch.  A query that sees no token at
 * all gives zeros.  A token that a query does not see does not reach it, whatever
 * its key and value hold; an infinity or NaN that it sees does.
 *
 *   page          tokens per page: 16, 32, 64, 128 or 256
 *   n_pages       pages of the caches
 *   q             bf16 [batch][steps][h_q][d]
 *   prefix_pages  int32 [ceil(prefix_len / page)]; null when prefix_len is 0
 *   prefix_len    tokens of the prefix, on the host (a step's launches do not
 *                 depend on the tails' lengths, so a captured step stays valid
 *                 while they grow)
 *   tail_pages    int32 [batch][tail_width], entries past a tail's end unread;
 *                 null when tail_width is 0 (no tails)
 *   tail_len      int32 [batch], device; null when tail_width is 0
 *   gate          null, or bf16 with element strides (token, head), multiples of
 *                 8, token = b * steps + i
 *   out           bf16 [batch][steps][h_q][d]
 *   workspace     >= gdn_attn_decode_shared_workspace_bytes, 256-byte aligned
 * A page index outside [0, n_pages) or a tail length outside
 * [0, tail_width * page] sets GDN_ERR_DEVICE_BOUNDS; the sequences that reach it
 * have unspecified outputs (nothing outside the caches is read).
 * Before it meets the values, each softmax weight is rounded to bf16, which moves out
 * by at most 2^-8 sum p |v| (times the gate's sigmoid) besides its own rounding;
 * everything else, the weights' sum among it, is fp32.
 * The order of a row's sums depends on the batch, the lengths and the GPU's SM
 * count, and on nothing else: equal calls give equal bits, but a sequence's last
 * bits may differ between batches.
 */
size_t gdn_attn_decode_shared_workspace_bytes(const gdn_attn_dims* dims, int batch, int steps);
gdn_status gdn_attn_decode_shared(const gdn_attn_dims* dims, int page, long long n_pages,
                                  int batch, int steps, const void* q, const void* k_cache,
                                  const void* v_cache, const int32_t* prefix_pages,
                                  long long prefix_len, const int32_t* tail_pages,
                                  int tail_width, const int32_t* tail_len, const void* gate,
                                  long long gate_token_stride, long long gate_head_stride,
                                  void* out, void* workspace, size_t workspace_bytes,
                                  int32_t* device_status, void* stream);

/*
 * A whole mixture-of-experts layer for a few tokens.  Per token x:
 *   p   = softmax(W_router x) over the experts
 *   top = the top_k largest (ties to the lowest index), weights p, divided by
 *         their sum when renorm is set
 *   y   = sum over top of weight_e W_down,e (silu(W_gate,e x) * (W_up,e x))
 *         + sigmoid(w_shared_gate . x) W_down,s (silu(W_gate,s x) * (W_up,s x))
 * the last line when shared_inter > 0 (without w_shared_gate its factor is 1).
 *
 *   x            bf16 [tokens][hidden], tokens 0 .. GDN_MOE_MAX_TOKENS
 *   w_router     bf16 [experts][hidden]
 *   w_gate_up    bf16 [experts][2 inter][hidden], the inter gate rows first
 *   w_down       bf16 [experts][hidden][inter]
 *   w_shared_gate_up [2 shared_inter][hidden], w_shared_down [hidden][shared_inter],
 *   w_shared_gate [hidden]: bf16; null when shared_inter is 0
 *   y            [tokens][hidden], bf16 or fp32 (out_dtype)
 *   topk_id      null or int32 [tokens][top_k];  topk_w null or fp32 [tokens][top_k]
 *   workspace    >= gdn_moe_step_workspace_bytes, 256-byte aligned
 * hidden, inter and shared_inter are multiples of 8, at most 16384; experts at
 * most 1024; top_k at most 32.  Router logits are compensated sums in pairs of
 * fp32: two logits are in their exact order when they are further apart than
 * 2 (hidden / 64 + 10)^2 2^-48 of the sum of their products' sizes (2^-36 at hidden
 * 2048; some 2^-45 as a rule), at any scale that fp32 holds.  A NaN logit is chosen
 * last; a token with a NaN or a positively infinite one has NaN for its weights and
 * its y, with renorm as without, as softmax gives them.  Everything else is
 * summed in fp32; the activations between the two products are carried as sums of
 * two bf16 (16 bits of significand) for a bf16 output and of three (24 bits) for an
 * fp32 output.  A token's result does not depend on the other tokens of the call,
 * bit for bit.
 */
typedef struct gdn_moe_dims {
  int hidden;
  int inter;
  int experts;
  int top_k;
  int shared_inter;
  int renorm;
} gdn_moe_dims;

#define GDN_MOE_MAX_TOKENS 64

size_t gdn_moe_step_workspace_bytes(const gdn_moe_dims* dims, int tokens);
gdn_status gdn_moe_step(const gdn_moe_dims* dims, int tokens, const void* x, const void* w_router,
                        const void* w_gate_up, const void* w_down, const void* w_shared_gate_up,
                        const void* w_shared_down, const void* w_shared_gate, void* y,
                        int out_dtype, int32_t* topk_id, float* topk_w, void* workspace,
                        size_t workspace_bytes, int32_t* device_status, void* stream);

/*
 * The attention layers' cache in 4 bits.  A quarter of the bytes of the bf16 cache and
 * an eighth of that again for scales: 4.5 bits a value.
 *   gdn_kv4_store        rows of k and v into the cache (after gdn_attn_prep's norms and
 *                        positions: its k_cache and v_cache arguments can be plain rows)
 *   gdn_kv4_load         rows out of it, as bf16 or fp32
 *   gdn_attn_decode_kv4  attention over it, a page table for each sequence
 *
 * Values.  The d channels of a token and head are held in groups of 32.  Of a group x
 * of bf16, with m its element of largest magnitude (the positive one where +m and -m
 * both occur), s = -m / 8 and code c = clamp(rint(x / s), -8, 7), ties to even; it
 * stands for s c, exactly.  A group whose |m| is below 2^-90 is held as zeros; one with
 * an infinity or a NaN in it reads back as NaN throughout.
 *
 * Cache.  uint8 [n_pages][h_kv][page / 16][18 d], page 16, 32, 64, 128 or 256 tokens;
 * cache row r = page_index * page + offset is one token.  16 tokens of a head are a unit
 * of 18 d bytes: 8 d of K codes, 8 d of V codes, and bf16 scales [token][d / 32 of K |
 * d / 32 of V].  Code + 8 is four bits; eight of them are a 32-bit word, and words stand
 * in 16-byte vectors [vector][32 lanes][4 words].  For token j of the unit and channel c,
 * word w = (j / 8) * (d / 32) + c / 32 is word w % 4 of vector w / 4, in
 *   K: lane (j % 8) * 4 + (c % 32) / 8, nibble (c % 8) / 2 + 4 (c % 2) (nibble 0 the lowest
 *      four bits), the whole word then rotated left by 3 bits;
 *   V: lane (c % 32) / 4 * 4 + (j % 8) / 2, nibble c % 4 + 4 (j % 2).
 * A row's bytes are its own: storing one leaves every other row as it was.
 */
size_t gdn_kv4_page_bytes(const gdn_attn_dims* dims, int page); /* 0 for invalid arguments */

/*
 *   tokens     rows in the list
 *   k, v       bf16, element strides (token, head), multiples of 8, the d elements of a
 *              head contiguous; null: that part of the rows stays as it is
 *   slot       int32 [tokens]: the cache row of each; negative: not stored (a load gives
 *              zeros).  Null: token t is row t.  A row at or past n_pages * page sets
 *              GDN_ERR_DEVICE_BOUNDS and counts as negative.  Rows to be stored have to
 *              differ: of two alike, each piece may be the one's or the other's.
 *   cache      as above, n_pages pages
 *   k_out, v_out  [tokens][h_kv][d], bf16 or fp32 per out_dtype; null: not wanted
 */
gdn_status gdn_kv4_store(const gdn_attn_dims* dims, int page, long long n_pages, long long tokens,
                         const void* k, long long k_token_stride, long long k_head_stride,
                         const void* v, long long v_token_stride, long long v_head_stride,
                         const int32_t* slot, void* cache, int32_t* device_status, void* stream);
gdn_status gdn_kv4_load(const gdn_attn_dims* dims, int page, long long n_pages, long long tokens,
                        const int32_t* slot, const void* cache, void* k_out, void* v_out,
                        int out_dtype, int32_t* device_status, void* stream);

/*
 * Attention of a batch over the 4-bit cache.  Sequence b holds len[b] tokens in the pages
 * that its row of the table names, the last `steps` of which are its query tokens
 * themselves: query i sees tokens 0 .. len[b] - steps + i.
 *   out = softmax(scale q K^T) V * sigmoid(gate)
 * A query that sees no token gives zeros.  A token that a query does not see does not
 * reach it, whatever the cache holds there; a NaN that it sees does.  Sequences may
 * share pages (a prefix's are then read from memory about once).
 *
 *   batch, steps  at most GDN_ATTN_MAX_BATCH and GDN_ATTN_MAX_STEPS; steps * h_q / h_kv
 *                 at most GDN_ATTN_MAX_ROWS
 *   q             bf16 [batch][steps][h_q][d]
 *   cache         as above
 *   table         int32 [batch][table_width], entries past a sequence's end of no account; null
 *                 when table_width is 0; table_width * page at most 2^30
 *   len           int32 [batch], device: a call's launches do not depend on the lengths,
 *                 so a captured step stays valid while they grow
 *   gate          null, or bf16 with element strides (token, head), multiples of 8,
 *                 token = b * steps + i
 *   out           bf16 [batch][steps][h_q][d]
 *   workspace     >= gdn_attn_decode_kv4_workspace_bytes, 256-byte aligned
 * A length outside [0, table_width * page] or a page index outside [0, n_pages) sets
 * GDN_ERR_DEVICE_BOUNDS: the sequence counts as empty, and the outputs of one that
 * reaches such a page are unspecified (nothing outside the cache is read).
 * Each softmax weight times its token's scale is rounded to fp16.  That moves a weight p by at
 * most 2^-11 p or, where p is below 2^-11 P, P the query's largest, by at most 2^-22 P (and no
 * more than p), whatever other queries see and other tokens and groups of channels hold.
 * Everything else is summed in fp32, with steps of the largest magnitude M in a value's group where
 * values cancel: at most 2^-16 sum p M of out, and of a score 2^-16 scale times the sum over its
 * groups of Q M, Q the query's largest magnitude (below 2^108).  Equal calls give equal bits; the
 * order of a row's sums, and with it the last bits, depends on the batch, the lengths,
 * table_width * page and the GPU's SM count.
 */
size_t gdn_attn_decode_kv4_workspace_bytes(const gdn_attn_dims* dims, int batch, int steps);
gdn_status gdn_attn_decode_kv4(const gdn_attn_dims* dims, int page, long long n_pages, int batch,
                               int steps, const void* q, const void* cache, const int32_t* table,
                               int table_width, const int32_t* len, const void* gate,
                               long long gate_token_stride, long long gate_head_stride, void* out,
                               void* workspace, size_t workspace_bytes, int32_t* device_status,
                               void* stream);

/*
 * The pool that cache pages come from (the source pages' "two-group paged pool", its group
 * of KV pages; the group of fixed states is gdn_state_copy's).  All its integers are
 * device arrays of the caller's, which the calls below keep in step with each other:
 *   refs   int32 [n_pages]          tables that hold the page; 0 (or less): it is free
 *   table  int32 [n_seqs][width]    each sequence's pages in order, entries past its end
 *                                   unread: what gdn_attn_decode_kv4 takes
 *   len    int32 [n_seqs]           tokens of each sequence
 * A pool starts as zeros; page: tokens of a page.  Every layer's cache whose rows follow the
 * same tables takes part in the copies: gdn_page_caches names up to GDN_PAGES_MAX_CACHES
 * arrays of n_pages pages, page_bytes[i] (a multiple of 16, at most 2^32) apart, 4-bit or
 * bf16 (K and V then are two); base and page_bytes are host arrays, read during the call.
 *
 *   extend   sequence seq[i] grows by count[i] tokens (0 .. steps; all by steps when count
 *            is null): pages are added as needed, and slot[i][j] is the cache row of its
 *            new token j (-1 for j >= count[i]), for gdn_attn_prep and gdn_kv4_store
 *   trim     sequence seq[i] keeps its first new_len[i] <= len tokens; where it then ends
 *            inside a page that other tables hold too, it gets a copy of its own
 *   fork     sequence dst[i], which holds no tokens, becomes what src[i] is when the call
 *            begins: whole pages are shared, a partly filled last one is copied.  A
 *            sequence may be forked several times in a call
 *   free     sequence seq[i] gives up all its pages and holds no tokens
 *   compact  pages in use move so that they are pages 0 .. n_live - 1 (each of those beyond
 *            to the lowest free one, in order) and every table follows; *n_live, if given, a
 *            device word, is set
 *   copy     page src_page[i] of every cache of one set to page dst_page[i] of another's
 *            (or the same), both in device memory: moving pages to another set and back; no
 *            pool is involved
 * Trimmed and freed sequences' entries become -1; a page whose count drops to 0 is free.
 * Pages that calls add are the lowest free ones, in the order of the list.  A page that is
 * not full belongs to one table alone (extend writes into it), which these calls see to.
 *
 *   seq, src, dst  int32 [n], device; a null seq is sequences 0 .. n - 1.  n at most n_seqs
 *                  and GDN_PAGES_MAX_LIST
 *   slot           int32 [n][steps]
 *   caches         null, or no arrays: the tables alone are changed
 *   workspace      >= gdn_pages_workspace_bytes, 256-byte aligned
 * extend, trim, fork and free are done whole or not at all: a sequence out of range or
 * named twice (as dst, of fork), a length or count that may not be, a fork into a sequence
 * that holds tokens, or too few free pages sets GDN_ERR_DEVICE_BOUNDS and changes
 * nothing (extend then gives -1 for all slots).  Free is what is free when the call begins, so a trim
 * that has to copy a shared page can be refused in a full pool, whatever it gives back itself;
 * one to a whole number of pages never is.  A page index out of range in a table or in copy's
 * lists sets GDN_ERR_DEVICE_BOUNDS too, but is only passed over.  copy's pairs run at the same time:
 * no destination may be another pair's, source or destination.
 */
#define GDN_PAGES_MAX_SEQS 65536
#define GDN_PAGES_MAX_LIST 8192
#define GDN_PAGES_MAX_CACHES 128

typedef struct gdn_page_pool {
  int n_pages;
  int page;
  int n_seqs;
  int width;
  int32_t* refs;
  int32_t* table;
  int32_t* len;
} gdn_page_pool;

typedef struct gdn_page_caches {
  int n;
  void* const* base;
  const size_t* page_bytes;
} gdn_page_caches;

size_t gdn_pages_workspace_bytes(const gdn_page_pool* pool);
gdn_status gdn_pages_extend(const gdn_page_pool* pool, const int32_t* seq, int n, int steps,
                            const int32_t* count, int32_t* slot, void* workspace,
                            size_t workspace_bytes, int32_t* device_status, void* stream);
gdn_status gdn_pages_trim(const gdn_page_pool* pool, const gdn_page_caches* caches,
                          const int32_t* seq, int n, const int32_t* new_len, void* workspace,
                          size_t workspace_bytes, int32_t* device_status, void* stream);
gdn_status gdn_pages_fork(const gdn_page_pool* pool, const gdn_page_caches* caches,
                          const int32_t* src, const int32_t* dst, int n, void* workspace,
                          size_t workspace_bytes, int32_t* device_status, void* stream);
gdn_status gdn_pages_free(const gdn_page_pool* pool, const int32_t* seq, int n, void* workspace,
                          size_t workspace_bytes, int32_t* device_status, void* stream);
gdn_status gdn_pages_compact(const gdn_page_pool* pool, const gdn_page_caches* caches,
                             int32_t* n_live, void* workspace, size_t workspace_bytes,
                             int32_t* device_status, void* stream);
gdn_status gdn_pages_copy(const gdn_page_caches* src, int src_pages, const int32_t* src_page,
                          const gdn_page_caches* dst, int dst_pages, const int32_t* dst_page, int n,
                          int32_t* device_status, void* stream);

/* Waits for the stream, then reads a device status word (the first 4 bytes
 * of a prefill workspace, or a decode device_status word) into *code:
 * GDN_OK or the first device-side error recorded.  Returns GDN_ERR_CUDA if
 * the copy or the wait failed. */
gdn_status gdn_read_device_status(const void* status_word, void* stream,
                                  int32_t* code);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
