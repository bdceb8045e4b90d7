// gdn_cache_api.cu -- the extern "C" surface of the 4-bit cache and of the pages' pool: validation and launch,
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

int log2_of(int page) {
  int n = 0;
  while (1 << n < page) ++n;
  return n;
}

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

gdn_status check_pool(const gdn_page_pool* p) {
  if (!p || p->n_pages < 0 || p->page < 1 || p->n_seqs < 0 || p->width < 0) return GDN_ERR_INVALID_ARG;
  if (p->n_seqs > GDN_PAGES_MAX_SEQS || p->n_pages > 0x7fffffff / p->page || p->width > 0x7fffffff / p->page)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// The pool's arrays and the workspace of a call that has something to do.
gdn_status check_pool_memory(const gdn_page_pool* p, const void* workspace, size_t workspace_bytes) {
  if ((p->n_pages > 0 && !p->refs) || (p->n_seqs > 0 && !p->len) || (p->n_seqs > 0 && p->width > 0 && !p->table) ||
      !maybe16(p->refs) || !maybe16(p->table) || !maybe16(p->len))
    return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < gdn::pages_scratch_bytes(p->n_pages, p->n_seqs))
    return GDN_ERR_WORKSPACE;
  return GDN_OK;
}

gdn_status check_list(const gdn_page_pool* p, const int32_t* seq, int n) {
  if (n < 0 || !maybe16(seq) || n > p->n_seqs) return GDN_ERR_INVALID_ARG;
  return n > GDN_PAGES_MAX_LIST ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

// Copies within one set of caches, or between two alike.
gdn_status check_caches(const gdn_page_caches* src, const gdn_page_caches* dst, gdn::PageMoves& m) {
  m = {};
  if (!src) return GDN_OK;
  if (src->n < 0 || (dst && dst->n != src->n)) return GDN_ERR_INVALID_ARG;
  if (src->n > GDN_PAGES_MAX_CACHES) return GDN_ERR_UNSUPPORTED;
  if (src->n > 0 && (!src->base || !src->page_bytes || (dst && (!dst->base || !dst->page_bytes))))
    return GDN_ERR_INVALID_ARG;
  long long pieces = 0;
  for (int i = 0; i < src->n; ++i) {
    const size_t bytes = src->page_bytes[i];
    if (!need16(src->base[i]) || (dst && (!need16(dst->base[i]) || dst->page_bytes[i] != bytes)) || bytes == 0 ||
        bytes % 16 != 0)
      return GDN_ERR_INVALID_ARG;
    if (bytes > (size_t(1) << 32)) return GDN_ERR_UNSUPPORTED;
    m.first[i] = (int)pieces;
    m.src[i] = static_cast<const uint8_t*>(src->base[i]);
    m.dst[i] = static_cast<uint8_t*>(dst ? dst->base[i] : src->base[i]);
    m.bytes[i] = (long long)bytes;
    pieces += gdn::page_pieces(bytes);
  }
  m.caches = src->n;
  m.first[m.caches] = (int)pieces;   // at most 128 * 2^20
  return GDN_OK;
}

gdn::PagePool pool_of(const gdn_page_pool* p) {
  return gdn::PagePool{p->n_pages, p->page, p->n_seqs, p->width, p->refs, p->table, p->len};
}

gdn_status launched(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

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
  p.page_log = log2_of(page);
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
  p.page_log = log2_of(page);
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
  if (table_width > (1 << 30) / page) return GDN_ERR_UNSUPPORTED;
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

size_t gdn_pages_workspace_bytes(const gdn_page_pool* pool) {
  if (check_pool(pool) != GDN_OK) return 0;
  return gdn::pages_scratch_bytes(pool->n_pages, pool->n_seqs);
}

gdn_status gdn_pages_extend(const gdn_page_pool* pool, const int32_t* seq, int n, int steps, const int32_t* count,
                            int32_t* slot, void* workspace, size_t workspace_bytes, int32_t* device_status,
                            void* stream) {
  gdn::TraceRange trace_range("gdn_pages_extend");
  gdn_status st = check_pool(pool);
  if (st == GDN_OK) st = check_list(pool, seq, n);
  if (st != GDN_OK) return st;
  if (steps < 0 || !aligned(device_status, 4) || !maybe16(count)) return GDN_ERR_INVALID_ARG;
  if (n == 0 || steps == 0) return GDN_OK;
  if (!need16(slot)) return GDN_ERR_INVALID_ARG;
  if ((st = check_pool_memory(pool, workspace, workspace_bytes)) != GDN_OK) return st;
  return launched(gdn::launch_pages_extend(pool_of(pool), gdn::PageList{seq, n}, steps, count, slot, workspace,
                                           device_status, static_cast<cudaStream_t>(stream)));
}

gdn_status gdn_pages_trim(const gdn_page_pool* pool, const gdn_page_caches* caches, const int32_t* seq, int n,
                          const int32_t* new_len, void* workspace, size_t workspace_bytes, int32_t* device_status,
                          void* stream) {
  gdn::TraceRange trace_range("gdn_pages_trim");
  gdn::PageMoves m;
  gdn_status st = check_pool(pool);
  if (st == GDN_OK) st = check_list(pool, seq, n);
  if (st == GDN_OK) st = check_caches(caches, nullptr, m);
  if (st != GDN_OK) return st;
  if (!aligned(device_status, 4)) return GDN_ERR_INVALID_ARG;
  if (n == 0) return GDN_OK;
  if (!need16(new_len)) return GDN_ERR_INVALID_ARG;
  if ((st = check_pool_memory(pool, workspace, workspace_bytes)) != GDN_OK) return st;
  return launched(gdn::launch_pages_trim(pool_of(pool), &m, gdn::PageList{seq, n}, new_len, workspace, device_status,
                                         static_cast<cudaStream_t>(stream)));
}

gdn_status gdn_pages_fork(const gdn_page_pool* pool, const gdn_page_caches* caches, const int32_t* src,
                          const int32_t* dst, int n, void* workspace, size_t workspace_bytes, int32_t* device_status,
                          void* stream) {
  gdn::TraceRange trace_range("gdn_pages_fork");
  gdn::PageMoves m;
  gdn_status st = check_pool(pool);
  if (st == GDN_OK) st = check_list(pool, dst, n);
  if (st == GDN_OK) st = check_caches(caches, nullptr, m);
  if (st != GDN_OK) return st;
  if (!aligned(device_status, 4)) return GDN_ERR_INVALID_ARG;
  if (n == 0) return GDN_OK;
  if (!need16(src) || !need16(dst)) return GDN_ERR_INVALID_ARG;
  if ((st = check_pool_memory(pool, workspace, workspace_bytes)) != GDN_OK) return st;
  return launched(gdn::launch_pages_fork(pool_of(pool), &m, src, dst, n, workspace, device_status,
                                         static_cast<cudaStream_t>(stream)));
}

gdn_status gdn_pages_free(const gdn_page_pool* pool, const int32_t* seq, int n, void* workspace,
                          size_t workspace_bytes, int32_t* device_status, void* stream) {
  gdn::TraceRange trace_range("gdn_pages_free");
  gdn_status st = check_pool(pool);
  if (st == GDN_OK) st = check_list(pool, seq, n);
  if (st != GDN_OK) return st;
  if (!aligned(device_status, 4)) return GDN_ERR_INVALID_ARG;
  if (n == 0) return GDN_OK;
  if ((st = check_pool_memory(pool, workspace, workspace_bytes)) != GDN_OK) return st;
  return launched(gdn::launch_pages_free(pool_of(pool), gdn::PageList{seq, n}, workspace, device_status,
                                         static_cast<cudaStream_t>(stream)));
}

gdn_status gdn_pages_compact(const gdn_page_pool* pool, const gdn_page_caches* caches, int32_t* n_live,
                             void* workspace, size_t workspace_bytes, int32_t* device_status, void* stream) {
  gdn::TraceRange trace_range("gdn_pages_compact");
  gdn::PageMoves m;
  gdn_status st = check_pool(pool);
  if (st == GDN_OK) st = check_caches(caches, nullptr, m);
  if (st != GDN_OK) return st;
  if (!aligned(device_status, 4) || !aligned(n_live, 4)) return GDN_ERR_INVALID_ARG;
  if (pool->n_pages == 0 && !n_live) return GDN_OK;
  if ((st = check_pool_memory(pool, workspace, workspace_bytes)) != GDN_OK) return st;
  return launched(gdn::launch_pages_compact(pool_of(pool), &m, n_live, workspace, device_status,
                                            static_cast<cudaStream_t>(stream)));
}

gdn_status gdn_pages_copy(const gdn_page_caches* src, int src_pages, const int32_t* src_page,
                          const gdn_page_caches* dst, int dst_pages, const int32_t* dst_page, int n,
                          int32_t* device_status, void* stream) {
  gdn::TraceRange trace_range("gdn_pages_copy");
  gdn::PageMoves m;
  if (!src || !dst) return GDN_ERR_INVALID_ARG;
  const gdn_status st = check_caches(src, dst, m);
  if (st != GDN_OK) return st;
  if (src_pages < 0 || dst_pages < 0 || n < 0 || !maybe16(src_page) || !maybe16(dst_page) ||
      !aligned(device_status, 4) || (!src_page && n > src_pages) || (!dst_page && n > dst_pages))
    return GDN_ERR_INVALID_ARG;
  if (n == 0 || m.caches == 0) return GDN_OK;
  m.from = src_page;
  m.to = dst_page;
  m.src_pages = src_pages;
  m.dst_pages = dst_pages;
  m.n = n;
  m.status = device_status;
  return launched(gdn::launch_pages_copy(m, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
