// gdn_moe.cu -- a whole mixture-of-experts layer for a few tokens.
//
// Four launches: router logits, top-k, gate/up products, down products with
// the sum over a token's experts.  A warp per dot product.
#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

// The dot product of two bf16 rows, good to about 48 bits.  S starts at a
// constant whose grid is coarser than any term's low part: each product's high
// part goes into S exactly, the rest (exact too, by the fused product) into lo.
__device__ __forceinline__ double dot_exact(const uint16_t* a, const uint16_t* b, int n, int lane) {
  const float C = 3072.0f;
  float S = C, lo = 0.0f;
  for (int i = lane; i < n; i += 32) {
    const float x = bf16_to_f32(a[i]), w = bf16_to_f32(b[i]);
    const float t = fmaf(x, w, S);
    const float d = t - S;
    S = t;
    lo += fmaf(x, w, -d);
  }
  double v = (double)(S - C) + (double)lo;
  for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

__device__ __forceinline__ float dot_bf16(const uint16_t* a, const uint16_t* b, int n, int lane) {
  float s = 0.0f;
  for (int i = lane; i < n; i += 32) s = fmaf(bf16_to_f32(a[i]), bf16_to_f32(b[i]), s);
  return warp_sum(s);
}

// e^x for x <= 0 given in 64 bits: the fp32 rounding of the argument is put
// back as a factor (at x = -80 it alone would cost 2^-18 of the result).
__device__ __forceinline__ float exp_of(double x) {
  const float h = (float)x;
  return h < -200.0f ? 0.0f : expf(h) * (1.0f + (float)(x - (double)h));
}

__global__ void router_kernel(const MoeArgs p, double* logit) {
  const int w = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (w >= p.tokens * p.experts) return;
  const int t = w / p.experts, e = w % p.experts;
  const double v = dot_exact(p.x + (size_t)t * p.hidden, p.w_router + (size_t)e * p.hidden, p.hidden, lane);
  if (lane == 0) logit[w] = v;
}

__global__ void topk_kernel(const MoeArgs p, double* logit, int* ids, float* wts) {
  const int t = blockIdx.x, lane = threadIdx.x;
  double* lg = logit + (size_t)t * p.experts;
  double top = -INFINITY;
  for (int e = lane; e < p.experts; e += 32) top = fmax(top, lg[e]);
  for (int m = 16; m >= 1; m >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, m));
  float den = 0.0f;
  for (int e = lane; e < p.experts; e += 32) den += exp_of(lg[e] - top);
  den = warp_sum(den);
  float sel = 0.0f;
  for (int k = 0; k < p.top_k; ++k) {
    double best = -INFINITY;
    int at = p.experts;
    for (int e = lane; e < p.experts; e += 32) {
      bool used = false;
      for (int j = 0; j < k; ++j) used |= ids[t * p.top_k + j] == e;
      if (!used && (at == p.experts || lg[e] > best)) { best = lg[e]; at = e; }
    }
    for (int m = 16; m >= 1; m >>= 1) {
      const double ob = __shfl_xor_sync(0xffffffffu, best, m);
      const int oa = __shfl_xor_sync(0xffffffffu, at, m);
      if (oa < p.experts && (at == p.experts || ob > best || (!(best > ob) && oa < at))) { best = ob; at = oa; }
    }
    const float w = exp_of(best - top) / den;
    sel += w;
    if (lane == 0) { ids[t * p.top_k + k] = at; wts[t * p.top_k + k] = w; }
    __syncwarp();
  }
  if (lane == 0)
    for (int k = 0; k < p.top_k; ++k) {
      float& w = wts[t * p.top_k + k];
      if (p.renorm) w /= sel;
      if (p.topk_id) p.topk_id[t * p.top_k + k] = ids[t * p.top_k + k];
      if (p.topk_w) p.topk_w[t * p.top_k + k] = w;
    }
}

__global__ void gate_up_kernel(const MoeArgs p, const int* ids, float* act, float* sact) {
  const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const long long routed = (long long)p.tokens * p.top_k * p.inter;
  const uint16_t* g;
  const uint16_t* x;
  int n;
  float* dst;
  if (w < routed) {
    const int i = (int)(w % p.inter), s = (int)(w / p.inter);
    g = p.w_gate_up + ((size_t)ids[s] * 2 * p.inter + i) * p.hidden;
    x = p.x + (size_t)(s / p.top_k) * p.hidden;
    n = p.inter;
    dst = act + w;
  } else {
    const long long v = w - routed;
    if (v >= (long long)p.tokens * p.shared_inter) return;
    g = p.s_gate_up + (size_t)(v % p.shared_inter) * p.hidden;
    x = p.x + (size_t)(v / p.shared_inter) * p.hidden;
    n = p.shared_inter;
    dst = sact + v;
  }
  const float a = dot_bf16(g, x, p.hidden, lane), b = dot_bf16(g + (size_t)n * p.hidden, x, p.hidden, lane);
  if (lane == 0) *dst = silu(a) * b;
}

__global__ void down_kernel(const MoeArgs p, const int* ids, const float* wts, const float* act, const float* sact) {
  const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= (long long)p.tokens * p.hidden) return;
  const int t = (int)(w / p.hidden), h = (int)(w % p.hidden);
  float y = 0.0f;
  for (int k = 0; k < p.top_k; ++k) {
    const int s = t * p.top_k + k;
    const uint16_t* d = p.w_down + ((size_t)ids[s] * p.hidden + h) * p.inter;
    float v = 0.0f;
    for (int i = lane; i < p.inter; i += 32) v = fmaf(bf16_to_f32(d[i]), act[(size_t)s * p.inter + i], v);
    y = fmaf(wts[s], warp_sum(v), y);
  }
  if (p.shared_inter) {
    float v = 0.0f;
    const uint16_t* d = p.s_down + (size_t)h * p.shared_inter;
    for (int i = lane; i < p.shared_inter; i += 32) v = fmaf(bf16_to_f32(d[i]), sact[(size_t)t * p.shared_inter + i], v);
    float f = 1.0f;
    if (p.s_gate) f = sigmoid(dot_bf16(p.s_gate, p.x + (size_t)t * p.hidden, p.hidden, lane));
    y = fmaf(f, warp_sum(v), y);
  }
  if (lane == 0) {
    if (p.out_f32)
      static_cast<float*>(p.y)[w] = y;
    else
      static_cast<uint16_t*>(p.y)[w] = f32_to_bf16(y);
  }
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

size_t moe_scratch_bytes(int tokens, int, int inter, int experts, int top_k, int shared_inter) {
  const size_t T = tokens > 0 ? tokens : 1;
  return up256(T * experts * 8) + 2 * up256(T * top_k * 4) + up256(T * top_k * inter * 4) +
         up256(T * shared_inter * 4) + 256;
}

cudaError_t launch_moe(const MoeArgs& p, cudaStream_t stream) {
  const size_t T = p.tokens;
  char* ws = static_cast<char*>(p.scratch);
  double* logit = reinterpret_cast<double*>(ws);
  ws += up256(T * p.experts * 8);
  int* ids = reinterpret_cast<int*>(ws);
  ws += up256(T * p.top_k * 4);
  float* wts = reinterpret_cast<float*>(ws);
  ws += up256(T * p.top_k * 4);
  float* act = reinterpret_cast<float*>(ws);
  ws += up256(T * p.top_k * p.inter * 4);
  float* sact = reinterpret_cast<float*>(ws);
  const auto grid = [](long long warps) { return (unsigned)((warps + 7) / 8); };
  router_kernel<<<grid((long long)T * p.experts), 256, 0, stream>>>(p, logit);
  topk_kernel<<<p.tokens, 32, 0, stream>>>(p, logit, ids, wts);
  gate_up_kernel<<<grid((long long)T * p.top_k * p.inter + (long long)T * p.shared_inter), 256, 0, stream>>>(
      p, ids, act, sact);
  down_kernel<<<grid((long long)T * p.hidden), 256, 0, stream>>>(p, ids, wts, act, sact);
  return cudaGetLastError();
}

}  // namespace gdn
