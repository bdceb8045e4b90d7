// gdn_attn_prep.cu -- q and k norms, rotary positions and the cache write of
// the attention layer, one pass over a token's heads (HBM-bound).
//
// Mathematics.  Per head x of q or k, y = x / sqrt(mean(x^2) + eps) * w, then
// each pair of the first `rot` dimensions is turned by phi = pos * inv_freq.
// The angle is kept as a fraction of a turn in 64-bit fixed point: F =
// frac(inv_freq / 2 pi) 2^64, and pos * F wraps modulo 2^64 exactly where the
// angle wraps modulo a turn, so the reduction of a far position costs one
// integer product and loses nothing (F is good to 2^-53, so at position 2^31
// the turn is good to 2^-24 or so; an fp32 product is off by a whole radian
// beyond 2^24).  The top 32 bits become the argument of sincospif.
//
// Layout.  A row of D elements is D/8 lanes of 16 bytes, so a warp holds 1, 2
// or 4 rows; the norm is a butterfly over the row's lanes and the partner of a
// pair half a rotation away is one shuffle away.  A warp takes one token (or a
// share of its heads, when the tokens alone cannot fill the GPU), computes the
// token's sines and cosines once and uses them for all of its heads.  Four
// rows are in flight per warp.
#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

constexpr int kPrepWarps = 8;
constexpr int kPrepBatch = 4;     // rows in flight per lane group
constexpr int kMaxFreq = 128;     // rot / 2 at d = 256

struct PrepShape {
  int nq, nk, nv;     // rows of a token: q heads, k heads, v heads
  int per_item;       // rows of one item, a multiple of the warp's rows
  int chunks;         // items per token
  long long items;
};

template <int D>
__global__ void __launch_bounds__(kPrepWarps * 32)
    attn_prep_kernel(const AttnPrepArgs p, const PrepShape sh) {
  constexpr int LPR = D / 8;        // lanes per row
  constexpr int RPW = 32 / LPR;     // rows per warp
  __shared__ uint64_t freq[kMaxFreq];
  __shared__ int axis[kMaxFreq];
  __shared__ float cosv[kPrepWarps][kMaxFreq], sinv[kPrepWarps][kMaxFreq];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPR, l = lane % LPR;
  const int nf = p.rot >> 1;
  for (int i = threadIdx.x; i < nf; i += blockDim.x) {
    const double turns = p.inv_freq[i] * 0.15915494309189533577;   // 1 / 2 pi
    const double frac = turns - floor(turns);
    freq[i] = __double2ull_rn(frac * 18446744073709551616.0);
    int ax = p.freq_axis ? p.freq_axis[i] : 0;
    if (ax < 0 || ax >= p.n_axes) {
      record_status(p.status, GDN_ERR_DEVICE_BOUNDS);
      ax = 0;
    }
    axis[i] = ax;
  }
  __syncthreads();

  const int rows = sh.nq + sh.nk + sh.nv;
  const long long stride = (long long)gridDim.x * kPrepWarps;
  for (long long it = (long long)blockIdx.x * kPrepWarps + warp; it < sh.items; it += stride) {
    long long t = it;
    int r_lo = 0;
    if (sh.chunks > 1) {   // items < 2^31 then
      t = (unsigned)it / (unsigned)sh.chunks;
      r_lo = (int)((unsigned)it % (unsigned)sh.chunks) * sh.per_item;
    }
    const int r_hi = min(rows, r_lo + sh.per_item);
    long long dst = t;
    if (p.slot && r_hi > sh.nq) {
      dst = p.slot[t];
      if (dst >= p.cache_rows) {
        record_status(p.status, GDN_ERR_DEVICE_BOUNDS);
        dst = -1;
      }
    }
    __syncwarp();
    for (int i = lane; i < nf; i += 32) {
      const long long pos = p.pos[(long long)axis[i] * p.tokens + t];
      const uint64_t turn = (uint64_t)pos * freq[i];
      // a signed fraction of a turn, [-1/2, 1/2), times 2: sin and cos of pi x
      sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &sinv[warp][i], &cosv[warp][i]);
    }
    __syncwarp();

    for (int r0 = r_lo; r0 < r_hi; r0 += RPW * kPrepBatch) {
      uint4 raw[kPrepBatch];
#pragma unroll
      for (int u = 0; u < kPrepBatch; ++u) {
        const int r = r0 + u * RPW + sub;
        if (r < r_hi) {
          const uint16_t* src;
          if (r < sh.nq)
            src = p.q + t * p.q_st + r * p.q_sh;
          else if (r < sh.nq + sh.nk)
            src = p.k + t * p.k_st + (r - sh.nq) * p.k_sh;
          else
            src = p.v + t * p.v_st + (r - sh.nq - sh.nk) * p.v_sh;
          raw[u] = *reinterpret_cast<const uint4*>(src + 8 * l);
        } else {
          raw[u] = make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int u = 0; u < kPrepBatch; ++u) {
        if (r0 + u * RPW >= r_hi) break;   // the whole warp
        const int r = r0 + u * RPW + sub;
        const bool is_q = r < sh.nq, is_v = r >= sh.nq + sh.nk;
        float y[8];
        {
          const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[2 * i] = __uint_as_float(w[i] << 16);
            y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
          }
        }
        const float* nw = is_q ? p.q_w : p.k_w;
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
        for (int m = LPR / 2; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        if (nw) {
          const float inv = rsqrtf(ss * (1.0f / D) + p.eps);
          const float4 w0 = __ldg(reinterpret_cast<const float4*>(nw) + 2 * l);
          const float4 w1 = __ldg(reinterpret_cast<const float4*>(nw) + 2 * l + 1);
          const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = y[i] * inv * w[i];
        }
        if (p.rot > 0) {
          if (p.pairs) {
            if (8 * l < p.rot) {
              const float4 c = *reinterpret_cast<const float4*>(&cosv[warp][4 * l]);
              const float4 s = *reinterpret_cast<const float4*>(&sinv[warp][4 * l]);
              const float cc[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float a = y[2 * i], b = y[2 * i + 1];
                y[2 * i] = a * cc[i] - b * sv[i];
                y[2 * i + 1] = b * cc[i] + a * sv[i];
              }
            }
          } else {
            // lanes 0 .. nf/8 - 1 hold the first of each pair, the next nf/8 the second
            const int nl = nf >> 3;
            const bool first = l < nl, turned = l < 2 * nl;
            const int from = sub * LPR + (first ? l + nl : turned ? l - nl : l);
            const int f = turned ? 8 * (first ? l : l - nl) : 0;
            const float4 c0 = *reinterpret_cast<const float4*>(&cosv[warp][f]);
            const float4 c1 = *reinterpret_cast<const float4*>(&cosv[warp][f + 4]);
            const float4 s0 = *reinterpret_cast<const float4*>(&sinv[warp][f]);
            const float4 s1 = *reinterpret_cast<const float4*>(&sinv[warp][f + 4]);
            const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            const float sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float o = __shfl_sync(0xffffffffu, y[i], from);
              if (turned) y[i] = first ? y[i] * cc[i] - o * sv[i] : y[i] * cc[i] + o * sv[i];
            }
          }
        }
        if (r < r_hi) {
          uint4 o = raw[u];
          if (!is_v) {
            o.x = pack_bf16x2(y[0], y[1]);
            o.y = pack_bf16x2(y[2], y[3]);
            o.z = pack_bf16x2(y[4], y[5]);
            o.w = pack_bf16x2(y[6], y[7]);
          }
          if (is_q) {
            *reinterpret_cast<uint4*>(p.q_out + (t * sh.nq + r) * D + 8 * l) = o;
          } else if (dst >= 0) {
            const int h = r - sh.nq - (is_v ? sh.nk : 0);
            uint16_t* c = is_v ? p.v_cache : p.k_cache;
            *reinterpret_cast<uint4*>(c + (dst * p.h_kv + h) * D + 8 * l) = o;
          }
        }
      }
    }
  }
}

template <int D>
cudaError_t launch_d(const AttnPrepArgs& p, cudaStream_t stream, int sms) {
  constexpr int RPW = 32 / (D / 8);
  PrepShape sh;
  sh.nq = p.q ? p.h_q : 0;
  sh.nk = p.k ? p.h_kv : 0;
  sh.nv = p.v ? p.h_kv : 0;
  const int rows = sh.nq + sh.nk + sh.nv;
  const int iters = (rows + RPW - 1) / RPW;   // warp iterations of a token
  // one token per warp when that gives every SM two rounds of 32 warps, else
  // shares of its heads down to one row per lane group
  const long long want = (long long)sms * 64;
  long long per = (p.tokens * iters + want - 1) / want;
  if (per < 1) per = 1;
  if (per > iters) per = iters;
  sh.per_item = (int)per * RPW;
  sh.chunks = (rows + sh.per_item - 1) / sh.per_item;
  sh.items = p.tokens * sh.chunks;
  const long long blocks = (sh.items + kPrepWarps - 1) / kPrepWarps;
  const long long cap = (long long)sms * 4;
  attn_prep_kernel<D><<<(unsigned)(blocks < cap ? blocks : cap), kPrepWarps * 32, 0, stream>>>(p, sh);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prep(const AttnPrepArgs& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  switch (p.d) {
    case 64: return launch_d<64>(p, stream, sms);
    case 128: return launch_d<128>(p, stream, sms);
    case 256: return launch_d<256>(p, stream, sms);
  }
  return cudaErrorInvalidValue;
}

}  // namespace gdn
