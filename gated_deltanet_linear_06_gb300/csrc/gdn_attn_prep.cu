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
// token's sines and cosines once and keeps its lanes' in registers for all of
// its heads.  Two rows per lane group are loaded while the two before them are
// turned, the next token's first ones included: without that the kernel waited
// for its loads more than it worked (262 us for 32768 tokens, 671 MB).
//
// Measured: 32768 tokens of 16 + 2 + 2 heads of 256 (671 MB) 119 us, 5.63 TB/s or
// 83 % of a plain copy's rate; 2049 tokens of 32 + 8 + 8 heads of 128 with three
// axes (50 MB) 16.1 us, where a warp has one or two rounds and their latency
// shows (18.4 before the launch passed under the kernel before it); 8 tokens 5 us,
// all latency, under a call that takes the host 10.
#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

constexpr int kPrepWarps = 8;
constexpr int kPrepBatch = 2;     // rows in flight per lane group, and as many ahead
constexpr int kMaxFreq = 128;     // rot / 2 at d = 256

struct PrepShape {
  int nq, nk, nv;     // rows of a token: q heads, k heads, v heads
  int per_item;       // rows of one item, a multiple of the warp's rows
  int chunks;         // items per token
  long long items;
};

template <int D, bool PAIRS>
__global__ void __launch_bounds__(kPrepWarps * 32, 3)
    attn_prep_kernel(const AttnPrepArgs p, const PrepShape sh) {
  constexpr int LPR = D / 8;        // lanes per row
  constexpr int RPW = 32 / LPR;     // rows per warp
  constexpr int STEP = RPW * kPrepBatch;
  __shared__ uint64_t freq[kMaxFreq];
  __shared__ int axis[kMaxFreq];
  __shared__ __align__(16) float cosv[kPrepWarps][kMaxFreq], sinv[kPrepWarps][kMaxFreq];
  __shared__ __align__(16) float norm_w[2][D];

  // launched as the kernel before it ends, whose results are there from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
  for (int i = threadIdx.x; i < D; i += blockDim.x) {
    norm_w[0][i] = p.q_w ? p.q_w[i] : 1.0f;
    norm_w[1][i] = p.k_w ? p.k_w[i] : 1.0f;
  }
  __syncthreads();
  // halves: lanes 0 .. nf/8 - 1 hold the first of each pair, the next nf/8 the second
  const int nl = nf >> 3;
  const bool first = l < nl, turned = PAIRS ? 8 * l < p.rot : l < 2 * nl;
  const int from = PAIRS || !turned ? lane : (first ? lane + nl : lane - nl);

  const int rows = sh.nq + sh.nk + sh.nv;
  const long long stride = (long long)gridDim.x * kPrepWarps;
  // one batch of rows of one item, [r, hi) of token t
  struct Place {
    long long it, t;
    int r, hi;
  };
  const auto enter = [&](Place& w) {
    w.t = w.it;
    w.r = 0;
    if (sh.chunks > 1) {   // items < 2^31 then
      w.t = (unsigned)w.it / (unsigned)sh.chunks;
      w.r = (int)((unsigned)w.it % (unsigned)sh.chunks) * sh.per_item;
    }
    w.hi = min(rows, w.r + sh.per_item);
  };
  const auto load = [&](uint4 (&raw)[kPrepBatch], const Place& w) {
    if (w.r + STEP <= sh.nq && w.r + STEP <= w.hi) {   // query heads only: most batches
      const uint16_t* src = p.q + w.t * p.q_st + (w.r + sub) * p.q_sh + 8 * l;
#pragma unroll
      for (int u = 0; u < kPrepBatch; ++u) raw[u] = *reinterpret_cast<const uint4*>(src + u * RPW * p.q_sh);
      return;
    }
#pragma unroll
    for (int u = 0; u < kPrepBatch; ++u) {
      const int r = w.r + u * RPW + sub;
      if (r < w.hi) {
        const uint16_t* src;
        if (r < sh.nq)
          src = p.q + w.t * p.q_st + r * p.q_sh;
        else if (r < sh.nq + sh.nk)
          src = p.k + w.t * p.k_st + (r - sh.nq) * p.k_sh;
        else
          src = p.v + w.t * p.v_st + (r - sh.nq - sh.nk) * p.v_sh;
        raw[u] = *reinterpret_cast<const uint4*>(src + 8 * l);
      } else {
        raw[u] = make_uint4(0, 0, 0, 0);
      }
    }
  };
  Place now;
  now.it = (long long)blockIdx.x * kPrepWarps + warp;
  if (now.it >= sh.items) return;
  enter(now);
  uint4 next[kPrepBatch];
  load(next, now);
  bool fresh = true;              // a new item: its angles and its cache row
  float c[PAIRS ? 4 : 8], s[PAIRS ? 4 : 8];
  long long dst = 0;
  while (true) {
    uint4 raw[kPrepBatch];
#pragma unroll
    for (int u = 0; u < kPrepBatch; ++u) raw[u] = next[u];
    Place then = now;
    then.r += STEP;
    const bool leave = then.r >= then.hi;
    if (leave) {
      then.it += stride;
      if (then.it < sh.items) enter(then);
    }
    const bool more = then.it < sh.items;
    if (more) load(next, then);
    if (fresh) {
      dst = now.t;
      if (p.slot && now.hi > sh.nq) {
        dst = p.slot[now.t];
        if (dst >= p.cache_rows) {
          record_status(p.status, GDN_ERR_DEVICE_BOUNDS);
          dst = -1;
        }
      }
      __syncwarp();
      for (int i = lane; i < nf; i += 32) {
        const long long pos = p.pos[(long long)axis[i] * p.tokens + now.t];
        const uint64_t turn = (uint64_t)pos * freq[i];
        // a signed fraction of a turn, [-1/2, 1/2), times 2: sin and cos of pi x
        sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &sinv[warp][i], &cosv[warp][i]);
      }
      __syncwarp();
      const int f = turned ? (PAIRS ? 4 * l : 8 * (first ? l : l - nl)) : 0;
#pragma unroll
      for (int i = 0; i < (PAIRS ? 4 : 8); i += 4) {
        const float4 cv = *reinterpret_cast<const float4*>(&cosv[warp][f + i]);
        const float4 sv = *reinterpret_cast<const float4*>(&sinv[warp][f + i]);
        const float sign = !PAIRS && first ? -1.0f : 1.0f;
        c[i] = cv.x, c[i + 1] = cv.y, c[i + 2] = cv.z, c[i + 3] = cv.w;
        s[i] = sign * sv.x, s[i + 1] = sign * sv.y, s[i + 2] = sign * sv.z, s[i + 3] = sign * sv.w;
      }
    }
    // one row: its norm with weights `nw` (null: none) and its rotation
    const auto turn_row = [&](const uint4& in, bool norm, const float* nw) -> uint4 {
      float y[8];
      {
        const uint32_t w[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[2 * i] = __uint_as_float(w[i] << 16);
          y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      }
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
      for (int m = LPR / 2; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      if (norm) {
        const float inv = rsqrtf(ss * (1.0f / D) + p.eps);
        const float4 w0 = *reinterpret_cast<const float4*>(nw + 8 * l);
        const float4 w1 = *reinterpret_cast<const float4*>(nw + 8 * l + 4);
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * inv * w[i];
      }
      if (nf > 0) {
        if (PAIRS) {
          if (turned) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float e = y[2 * i], o = y[2 * i + 1];
              y[2 * i] = e * c[i] - o * s[i];
              y[2 * i + 1] = o * c[i] + e * s[i];
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float o = __shfl_sync(0xffffffffu, y[i], from);
            const float v = y[i] * c[i % (PAIRS ? 4 : 8)] + o * s[i % (PAIRS ? 4 : 8)];
            y[i] = turned ? v : y[i];
          }
        }
      }
      return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                        pack_bf16x2(y[6], y[7]));
    };
    if (now.r + STEP <= sh.nq && now.r + STEP <= now.hi) {   // query heads only
      uint16_t* out = p.q_out + (now.t * sh.nq + now.r + sub) * D + 8 * l;
#pragma unroll
      for (int u = 0; u < kPrepBatch; ++u)
        *reinterpret_cast<uint4*>(out + u * RPW * D) = turn_row(raw[u], p.q_w != nullptr, norm_w[0]);
    } else {
#pragma unroll
      for (int u = 0; u < kPrepBatch; ++u) {
        if (now.r + u * RPW >= now.hi) break;   // the whole warp
        const int r = now.r + u * RPW + sub;
        const bool is_q = r < sh.nq, is_v = r >= sh.nq + sh.nk;
        uint4 o = raw[u];
        if (now.r + u * RPW < sh.nq + sh.nk) {  // (values alone: the whole warp)
          const uint4 y = turn_row(raw[u], is_q ? p.q_w != nullptr : p.k_w != nullptr, norm_w[is_q ? 0 : 1]);
          if (!is_v) o = y;
        }
        if (r < now.hi) {
          if (is_q) {
            *reinterpret_cast<uint4*>(p.q_out + (now.t * sh.nq + r) * D + 8 * l) = o;
          } else if (dst >= 0) {
            const int h = r - sh.nq - (is_v ? sh.nk : 0);
            uint16_t* cache = is_v ? p.v_cache : p.k_cache;
            *reinterpret_cast<uint4*>(cache + (dst * p.h_kv + h) * D + 8 * l) = o;
          }
        }
      }
    }
    if (!more) break;
    fresh = leave;
    now = then;
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
  // shares of its heads down to one row per lane group (choosing the share that
  // fills whole rounds best made no difference at 2049 tokens: 16.4 us both)
  const long long want = (long long)sms * 64;
  long long per = (p.tokens * iters + want - 1) / want;
  if (per < 1) per = 1;
  if (per > iters) per = iters;
  sh.per_item = (int)per * RPW;
  sh.chunks = (rows + sh.per_item - 1) / sh.per_item;
  sh.items = p.tokens * sh.chunks;
  const long long blocks = (sh.items + kPrepWarps - 1) / kPrepWarps;
  const long long cap = (long long)sms * 3;
  const unsigned grid = (unsigned)(blocks < cap ? blocks : cap);
  cudaLaunchAttribute overlap;
  overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  overlap.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kPrepWarps * 32);
  cfg.stream = stream;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, p.pairs ? attn_prep_kernel<D, true> : attn_prep_kernel<D, false>, p, sh);
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
