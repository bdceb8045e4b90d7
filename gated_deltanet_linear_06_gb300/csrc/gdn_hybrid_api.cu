// gdn_hybrid_api.cu -- the extern "C" surface of the attention layer's and the
// expert layer's operators: validation and launch, on the same terms as
// gdn_api.cu (nothing is launched and nothing touched on a refused argument).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/gdn.h"
#include "gdn_launch.h"
#include "gdn_trace.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool need16(const void* p) { return p != nullptr && aligned(p, 16); }
bool maybe16(const void* p) { return aligned(p, 16); }

gdn_status check_attn(const gdn_attn_dims* d) {
  if (!d || d->h_q <= 0 || d->h_kv <= 0 || d->h_q % d->h_kv != 0 || d->d <= 0 || d->rot < 0 ||
      d->rot > d->d || d->n_axes < 1 || !isfinite(d->norm_eps) || d->norm_eps < 0.0f ||
      !isfinite(d->scale) || d->scale < 0.0f || (d->rope_pairs != 0 && d->rope_pairs != 1))
    return GDN_ERR_INVALID_ARG;
  if ((d->d != 64 && d->d != 128 && d->d != 256) || d->rot % 16 != 0 ||
      d->n_axes > GDN_ATTN_MAX_AXES || d->h_q > 1024)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// A strided [token][head][d] input: 16-byte rows.
bool strides_ok(long long st, long long sh) { return st >= 0 && sh >= 0 && st % 8 == 0 && sh % 8 == 0; }

gdn_status check_shared(const gdn_attn_dims* d, int batch, int steps) {
  gdn_status st = check_attn(d);
  if (st != GDN_OK) return st;
  if (batch < 0 || steps < 1) return GDN_ERR_INVALID_ARG;
  if (batch > GDN_ATTN_MAX_BATCH || steps > GDN_ATTN_MAX_STEPS ||
      steps * (d->h_q / d->h_kv) > GDN_ATTN_MAX_ROWS)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

gdn_status check_moe(const gdn_moe_dims* d, int tokens) {
  if (!d || d->hidden <= 0 || d->inter <= 0 || d->experts <= 0 || d->top_k <= 0 ||
      d->top_k > d->experts || d->shared_inter < 0 || tokens < 0)
    return GDN_ERR_INVALID_ARG;
  if (d->hidden % 8 || d->inter % 8 || d->shared_inter % 8 || d->hidden > 16384 || d->inter > 16384 ||
      d->shared_inter > 16384 || d->experts > 1024 || d->top_k > 32 || tokens > GDN_MOE_MAX_TOKENS)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_attn_prep(const gdn_attn_dims* dims, long long tokens, const void* q,
                         long long q_token_stride, long long q_head_stride, const void* k,
                         long long k_token_stride, long long k_head_stride, const void* v,
                         long long v_token_stride, long long v_head_stride,
                         const float* q_norm_w, const float* k_norm_w, const double* inv_freq,
                         const int32_t* freq_axis, const int32_t* pos, const int32_t* slot,
                         long long cache_rows, void* q_out, void* k_cache, void* v_cache,
                         int32_t* device_status, void* stream) {
  gdn::TraceRange trace_range("gdn_attn_prep");
  const gdn_status st = check_attn(dims);
  if (st != GDN_OK) return st;
  if (tokens < 0 || tokens > 0x7fffffffLL || cache_rows < 0 || !aligned(device_status, 4))
    return GDN_ERR_INVALID_ARG;
  if (tokens == 0 || (!q && !k && !v)) return GDN_OK;
  if (!maybe16(q) || !maybe16(k) || !maybe16(v) || !maybe16(q_norm_w) || !maybe16(k_norm_w) ||
      !maybe16(slot) || !maybe16(freq_axis))
    return GDN_ERR_INVALID_ARG;
  if ((q && (!need16(q_out) || !strides_ok(q_token_stride, q_head_stride))) ||
      (k && (!need16(k_cache) || !strides_ok(k_token_stride, k_head_stride))) ||
      (v && (!need16(v_cache) || !strides_ok(v_token_stride, v_head_stride))))
    return GDN_ERR_INVALID_ARG;
  if (!slot && (k || v) && tokens > cache_rows) return GDN_ERR_INVALID_ARG;
  if (dims->rot > 0 && (q || k) &&
      (!need16(inv_freq) || !need16(pos) || (dims->n_axes > 1 && !freq_axis)))
    return GDN_ERR_INVALID_ARG;
  gdn::AttnPrepArgs p;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_st = q_token_stride;
  p.q_sh = q_head_stride;
  p.k_st = k_token_stride;
  p.k_sh = k_head_stride;
  p.v_st = v_token_stride;
  p.v_sh = v_head_stride;
  p.q_w = q_norm_w;
  p.k_w = k_norm_w;
  p.inv_freq = inv_freq;
  p.freq_axis = dims->n_axes > 1 ? freq_axis : nullptr;
  p.pos = pos;
  p.slot = slot;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_cache = static_cast<uint16_t*>(k_cache);
  p.v_cache = static_cast<uint16_t*>(v_cache);
  p.status = device_status;
  p.tokens = tokens;
  p.cache_rows = cache_rows;
  p.h_q = dims->h_q;
  p.h_kv = dims->h_kv;
  p.d = dims->d;
  p.rot = (q || k) ? dims->rot : 0;
  p.n_axes = dims->n_axes;
  p.pairs = dims->rope_pairs;
  p.eps = dims->norm_eps;
  return gdn::launch_attn_prep(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK
                                                                                    : GDN_ERR_CUDA;
}

size_t gdn_attn_decode_shared_workspace_bytes(const gdn_attn_dims* dims, int batch, int steps) {
  if (check_shared(dims, batch, steps) != GDN_OK) return 0;
  return gdn::attn_shared_scratch_bytes(batch, steps, dims->h_q, dims->h_kv, dims->d);
}

gdn_status gdn_attn_decode_shared(const gdn_attn_dims* dims, int page, long long n_pages,
                                  int batch, int steps, const void* q, const void* k_cache,
                                  const void* v_cache, const int32_t* prefix_pages,
                                  long long prefix_len, const int32_t* tail_pages,
                                  int tail_width, const int32_t* tail_len, const void* gate,
                                  long long gate_token_stride, long long gate_head_stride,
                                  void* out, void* workspace, size_t workspace_bytes,
                                  int32_t* device_status, void* stream) {
  gdn::TraceRange trace_range("gdn_attn_decode_shared");
  const gdn_status st = check_shared(dims, batch, steps);
  if (st != GDN_OK) return st;
  if (page <= 0 || n_pages < 0 || n_pages > (1LL << 40) || prefix_len < 0 || tail_width < 0 || !aligned(device_status, 4))
    return GDN_ERR_INVALID_ARG;
  if (page != 16 && page != 32 && page != 64 && page != 128 && page != 256) return GDN_ERR_UNSUPPORTED;
  if (prefix_len > 0x7fffffffLL || n_pages * page > 0x7fffffffLL || (long long)tail_width * page > 0x7fffffffLL)
    return GDN_ERR_UNSUPPORTED;
  if (batch == 0) return GDN_OK;
  if (!need16(q) || !need16(out) || !maybe16(gate) || !maybe16(prefix_pages) || !maybe16(tail_pages) ||
      !maybe16(tail_len))
    return GDN_ERR_INVALID_ARG;
  if ((prefix_len > 0 && !prefix_pages) || (tail_width > 0 && (!tail_pages || !tail_len)))
    return GDN_ERR_INVALID_ARG;
  if ((prefix_len > 0 || tail_width > 0) && (!need16(k_cache) || !need16(v_cache) || n_pages < 1))
    return GDN_ERR_INVALID_ARG;
  if (gate && !strides_ok(gate_token_stride, gate_head_stride)) return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < gdn::attn_shared_scratch_bytes(batch, steps, dims->h_q, dims->h_kv, dims->d))
    return GDN_ERR_WORKSPACE;
  gdn::AttnSharedArgs p;
  p.q = static_cast<const uint16_t*>(q);
  p.k_cache = static_cast<const uint16_t*>(k_cache);
  p.v_cache = static_cast<const uint16_t*>(v_cache);
  p.gate = static_cast<const uint16_t*>(gate);
  p.prefix_pages = prefix_pages;
  p.tail_pages = tail_pages;
  p.tail_len = tail_len;
  p.prefix_len = prefix_len;
  p.n_pages = n_pages;
  p.gate_st = gate_token_stride;
  p.gate_sh = gate_head_stride;
  p.out = static_cast<uint16_t*>(out);
  p.scratch = workspace;
  p.status = device_status;
  p.batch = batch;
  p.steps = steps;
  p.h_q = dims->h_q;
  p.h_kv = dims->h_kv;
  p.d = dims->d;
  p.page = page;
  p.tail_width = tail_width;
  p.scale = dims->scale > 0.0f ? dims->scale : 1.0f / sqrtf((float)dims->d);
  return gdn::launch_attn_shared(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK
                                                                                      : GDN_ERR_CUDA;
}

size_t gdn_moe_step_workspace_bytes(const gdn_moe_dims* dims, int tokens) {
  if (check_moe(dims, tokens) != GDN_OK) return 0;
  return gdn::moe_scratch_bytes(tokens, dims->hidden, dims->inter, dims->experts, dims->top_k,
                                dims->shared_inter);
}

gdn_status gdn_moe_step(const gdn_moe_dims* dims, int tokens, const void* x, const void* w_router,
                        const void* w_gate_up, const void* w_down, const void* w_shared_gate_up,
                        const void* w_shared_down, const void* w_shared_gate, void* y,
                        int out_dtype, int32_t* topk_id, float* topk_w, void* workspace,
                        size_t workspace_bytes, int32_t* device_status, void* stream) {
  gdn::TraceRange trace_range("gdn_moe_step");
  const gdn_status st = check_moe(dims, tokens);
  if (st != GDN_OK) return st;
  if ((out_dtype != GDN_DTYPE_BF16 && out_dtype != GDN_DTYPE_F32) || !aligned(device_status, 4))
    return GDN_ERR_INVALID_ARG;
  if (tokens == 0) return GDN_OK;
  if (!need16(x) || !need16(w_router) || !need16(w_gate_up) || !need16(w_down) || !need16(y) ||
      !maybe16(topk_id) || !maybe16(topk_w))
    return GDN_ERR_INVALID_ARG;
  if (dims->shared_inter > 0 &&
      (!need16(w_shared_gate_up) || !need16(w_shared_down) || !maybe16(w_shared_gate)))
    return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < gdn_moe_step_workspace_bytes(dims, tokens))
    return GDN_ERR_WORKSPACE;
  gdn::MoeArgs p;
  p.x = static_cast<const uint16_t*>(x);
  p.w_router = static_cast<const uint16_t*>(w_router);
  p.w_gate_up = static_cast<const uint16_t*>(w_gate_up);
  p.w_down = static_cast<const uint16_t*>(w_down);
  p.s_gate_up = static_cast<const uint16_t*>(w_shared_gate_up);
  p.s_down = static_cast<const uint16_t*>(w_shared_down);
  p.s_gate = static_cast<const uint16_t*>(w_shared_gate);
  p.y = y;
  p.topk_id = topk_id;
  p.topk_w = topk_w;
  p.scratch = workspace;
  p.status = device_status;
  p.tokens = tokens;
  p.hidden = dims->hidden;
  p.inter = dims->inter;
  p.experts = dims->experts;
  p.top_k = dims->top_k;
  p.shared_inter = dims->shared_inter;
  p.renorm = dims->renorm != 0;
  p.out_f32 = out_dtype == GDN_DTYPE_F32;
  return gdn::launch_moe(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
