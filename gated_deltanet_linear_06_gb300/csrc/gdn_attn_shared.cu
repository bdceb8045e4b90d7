// gdn_attn_shared.cu -- attention of a batch of sequences that share a prefix.
//
// One CTA per (query row, head), four warps that take every fourth key: the
// running maximum, sum and output of the softmax per warp, joined at the end.
#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

template <int D>
__global__ void __launch_bounds__(128) attn_shared_simple(const AttnSharedArgs p) {
  constexpr int E = D / 32;
  const int tok = blockIdx.x, h = blockIdx.y, b = tok / p.steps, step = tok % p.steps;
  const int hk = h / (p.h_q / p.h_kv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float so[4][D], sm[4], sl[4];
  float q[E], o[E], m = -INFINITY, den = 0.0f;
  for (int e = 0; e < E; ++e) {
    q[e] = bf16_to_f32(p.q[((size_t)tok * p.h_q + h) * D + e * 32 + lane]) * p.scale;
    o[e] = 0.0f;
  }
  long long tail = p.tail_width > 0 ? p.tail_len[b] : 0;
  if (tail < 0 || tail > (long long)p.tail_width * p.page) {
    record_status(p.status, GDN_ERR_DEVICE_BOUNDS);
    tail = 0;
  }
  const long long seen = max(0LL, tail - p.steps + 1 + step);
  for (long long j = warp; j < p.prefix_len + seen; j += 4) {
    const bool pre = j < p.prefix_len;
    const long long jj = pre ? j : j - p.prefix_len;
    const long long pg = pre ? p.prefix_pages[jj / p.page] : p.tail_pages[(size_t)b * p.tail_width + jj / p.page];
    if (pg < 0 || pg >= p.n_pages) {
      record_status(p.status, GDN_ERR_DEVICE_BOUNDS);
      continue;
    }
    const size_t row = ((size_t)(pg * p.page + jj % p.page) * p.h_kv + hk) * D;
    float s = 0.0f;
    for (int e = 0; e < E; ++e) s = fmaf(q[e], bf16_to_f32(p.k_cache[row + e * 32 + lane]), s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s);
    if (mn == -INFINITY) continue;
    const float c = __expf(m - mn), w = __expf(s - mn);
    den = den * c + w;
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + w * bf16_to_f32(p.v_cache[row + e * 32 + lane]);
    m = mn;
  }
  for (int e = 0; e < E; ++e) so[warp][e * 32 + lane] = o[e];
  if (lane == 0) { sm[warp] = m; sl[warp] = den; }
  __syncthreads();
  const float mt = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  for (int i = threadIdx.x; i < D; i += 128) {
    float a = 0.0f, l = 0.0f;
    for (int w = 0; w < 4; ++w) {
      const float c = sm[w] == -INFINITY ? 0.0f : __expf(sm[w] - mt);
      a += c * so[w][i];
      l += c * sl[w];
    }
    float r = l > 0.0f ? a / l : (l == 0.0f ? 0.0f : l);
    if (p.gate) r *= sigmoid(bf16_to_f32(p.gate[(size_t)tok * p.gate_st + (size_t)h * p.gate_sh + i]));
    p.out[((size_t)tok * p.h_q + h) * D + i] = f32_to_bf16(r);
  }
}

}  // namespace

size_t attn_shared_scratch_bytes(int, int, int, int, int) { return 256; }

cudaError_t launch_attn_shared(const AttnSharedArgs& p, cudaStream_t stream) {
  const dim3 grid(p.batch * p.steps, p.h_q);
  switch (p.d) {
    case 64: attn_shared_simple<64><<<grid, 128, 0, stream>>>(p); break;
    case 128: attn_shared_simple<128><<<grid, 128, 0, stream>>>(p); break;
    case 256: attn_shared_simple<256><<<grid, 128, 0, stream>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace gdn
