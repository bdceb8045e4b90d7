// gdn_cache_api.cu -- the extern "C" surface of the 4-bit cache: validation and launch,
// on the same terms as gdn_api.cu (nothing is launched and nothing touched on a refused
// argument).
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

bool page_size(int page) { return page == 16 || page == 32 || page == 64 || page == 128 || page == 256; }

// What these calls take of the attention dimensions: heads, head size, scale.
gdn_status check_dims(const gdn_attn_dims* d) {
  if (!d || d->h_q <= 0 || d->h_kv <= 0 || d->h_q % d->h_kv != 0 || d->d <= 0 || !isfinite(d->scale) ||
      d->scale < 0.0f)
    return GDN_ERR_INVALID_ARG;
  if ((d->d != 64 && d->d != 128 && d->d != 256) || d->h_q > 1024) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

gdn_status check_cache(int page, long long n_pages) {
  if (page <= 0 || n_pages < 0) return GDN_ERR_INVALID_ARG;
  if (!page_size(page) || n_pages > 0x7fffffffLL / page) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

bool strides_ok(long long st, long long sh) { return st >= 0 && sh >= 0 && st % 8 == 0 && sh % 8 == 0; }

gdn_status check_decode(const gdn_attn_dims* d, int batch, int steps) {
  const gdn_status st = check_dims(d);
  if (st != GDN_OK) return st;
  if (batch < 0 || steps < 1) return GDN_ERR_INVALID_ARG;
  if (batch > GDN_ATTN_MAX_BATCH || steps > GDN_ATTN_MAX_STEPS || steps * (d->h_q / d->h_kv) > GDN_ATTN_MAX_ROWS)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_kv4_page_bytes(const gdn_attn_dims* dims, int page) {
  if (check_dims(dims) != GDN_OK || !page_size(page)) return 0;
  return (size_t)page / 16 * 18 * dims->d * dims->h_kv;
}

gdn_status gdn_kv4_store(const gdn_attn_dims* dims, int page, long long n_pages, long long tokens,
                         const void* k, long long k_token_stride, long long k_head_stride,
                         const void* v, long long v_token_stride, long long v_head_stride,
                         const int32_t* slot, void* cache, int32_t* device_status, void* stream) {
  gdn::TraceRange trace_range("gdn_kv4_store");
  gdn_status st = check_dims(dims);
  if (st == GDN_OK) st = check_cache(page, n_pages);
  if (st != GDN_OK) return st;
  if (tokens < 0 || tokens > 0x7fffffffLL || !aligned(device_status, 4)) return GDN_ERR_INVALID_ARG;
  if (tokens == 0 || (!k && !v)) return GDN_OK;
  if (!maybe16(k) || !maybe16(v) || !maybe16(slot) || !need16(cache) || (k && !strides_ok(k_token_stride, k_head_stride)) ||
      (v && !strides_ok(v_token_stride, v_head_stride)) || (!slot && tokens > n_pages * page))
    return GDN_ERR_INVALID_ARG;
  gdn::Kv4RowsArgs p = {};
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.k_st = k_token_stride;
  p.k_sh = k_head_stride;
  p.v_st = v_token_stride;
  p.v_sh = v_head_stride;
  p.slot = slot;
  p.cache = static_cast<uint8_t*>(cache);
  p.status = device_status;
  p.tokens = tokens;
  p.cache_rows = n_pages * page;
  p.h_kv = dims->h_kv;
  p.d = dims->d;
  p.page = page;
  return gdn::launch_kv4_store(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_kv4_load(const gdn_attn_dims* dims, int page, long long n_pages, long long tokens,
                        const int32_t* slot, const void* cache, void* k_out, void* v_out,
                        int out_dtype, int32_t* device_status, void* stream) {
  gdn::TraceRange trace_range("gdn_kv4_load");
  gdn_status st = check_dims(dims);
  if (st == GDN_OK) st = check_cache(page, n_pages);
  if (st != GDN_OK) return st;
  if (tokens < 0 || tokens > 0x7fffffffLL || (out_dtype != GDN_DTYPE_BF16 && out_dtype != GDN_DTYPE_F32) ||
      !aligned(device_status, 4))
    return GDN_ERR_INVALID_ARG;
  if (tokens == 0 || (!k_out && !v_out)) return GDN_OK;
  if (!maybe16(k_out) || !maybe16(v_out) || !maybe16(slot) || !need16(cache) || (!slot && tokens > n_pages * page))
    return GDN_ERR_INVALID_ARG;
  gdn::Kv4RowsArgs p = {};
  p.k = static_cast<const uint16_t*>(k_out);
  p.v = static_cast<const uint16_t*>(v_out);
  p.slot = slot;
  p.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  p.k_out = k_out;
  p.v_out = v_out;
  p.status = device_status;
  p.tokens = tokens;
  p.cache_rows = n_pages * page;
  p.h_kv = dims->h_kv;
  p.d = dims->d;
  p.page = page;
  p.out_f32 = out_dtype == GDN_DTYPE_F32;
  return gdn::launch_kv4_load(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_attn_decode_kv4_workspace_bytes(const gdn_attn_dims* dims, int batch, int steps) {
  if (check_decode(dims, batch, steps) != GDN_OK) return 0;
  return gdn::attn_kv4_scratch_bytes(batch, steps, dims->h_q, dims->h_kv, dims->d);
}

gdn_status gdn_attn_decode_kv4(const gdn_attn_dims* dims, int page, long long n_pages, int batch,
                               int steps, const void* q, const void* cache, const int32_t* table,
                               int table_width, const int32_t* len, const void* gate,
                               long long gate_token_stride, long long gate_head_stride, void* out,
                               void* workspace, size_t workspace_bytes, int32_t* device_status,
                               void* stream) {
  gdn::TraceRange trace_range("gdn_attn_decode_kv4");
  gdn_status st = check_decode(dims, batch, steps);
  if (st == GDN_OK) st = check_cache(page, n_pages);
  if (st != GDN_OK) return st;
  if (table_width < 0 || !aligned(device_status, 4)) return GDN_ERR_INVALID_ARG;
  if (table_width > 0x7fffffffLL / page) return GDN_ERR_UNSUPPORTED;
  if (batch == 0) return GDN_OK;
  if (!need16(q) || !need16(out) || !need16(len) || !maybe16(gate) || !maybe16(table) ||
      (table_width > 0 && (!table || !need16(cache) || n_pages < 1)) ||
      (gate && !strides_ok(gate_token_stride, gate_head_stride)))
    return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < gdn::attn_kv4_scratch_bytes(batch, steps, dims->h_q, dims->h_kv, dims->d))
    return GDN_ERR_WORKSPACE;
  gdn::AttnKv4Args p;
  p.q = static_cast<const uint16_t*>(q);
  p.gate = static_cast<const uint16_t*>(gate);
  p.cache = static_cast<const uint8_t*>(cache);
  p.table = table;
  p.len = len;
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
  p.width = table_width;
  p.scale = dims->scale > 0.0f ? dims->scale : 1.0f / sqrtf((float)dims->d);
  return gdn::launch_attn_kv4(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
