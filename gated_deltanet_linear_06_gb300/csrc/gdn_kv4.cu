// gdn_kv4.cu -- rows of k and v into the 4-bit cache (gdn_kv4_store) and back out of it
// (gdn_kv4_load).
//
// Both are streams: a row is read once and written once.  The work is cut the way the cache's
// vectors lie.  A warp of a store takes sixteen tokens of the list, one head, K or V and a
// 16-byte vector per lane: four lanes read 32 channels of a token, find the group's scale
// between them and make K's vector as it stands; V's vectors hold two tokens' channels and are
// put together between lanes where the tokens are a unit's in order.  Elsewhere (a decode
// step's rows, one of each sequence) V's pieces are two bytes each.  A list that runs through
// units need not begin with one: the tokens are taken in sixteens that end where the first
// token's unit does.
//
// A store takes some 16 instructions a value (of which 5 for the quotient, its rounding and its
// place), less than half of what they were with divisions and without extremes as packed 16-bit
// numbers.  Nothing that it uses is full (issue slots 68 %, integer pipe 61 %, memory 63 %): a warp
// loads its vectors, converts them, stores them and ends, so that loads and arithmetic overlap
// between warps only.  Measured, 32768 rows of 2 heads of 256: store 20.7 us (4.2 TB/s of 67 MB
// read and 19 MB written), load as bf16 15 us (5.8 TB/s).  256 rows of as many
// sequences: 5 us each, latency.
#include "../../include/gdn.h"
#include "gdn_kv4.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

constexpr int kKv4Warps = 8;

// One warp's share of a call: tokens first .. first + 15 of the list (those in range),
// head, K or V, vector.
struct Share {
  long long first;
  int head, vec;
  bool is_v;
};

template <int D>
__device__ __forceinline__ bool share_of(const Kv4RowsArgs& p, unsigned item, int vectors, Share& s) {
  const int NV = D / 64 / vectors;
  const unsigned kinds = (p.k != nullptr) + (p.v != nullptr);
  const unsigned per = p.h_kv * kinds * NV, block = item / per;
  unsigned rest = item - block * per;
  s.vec = rest % NV * vectors;
  rest /= NV;
  s.is_v = p.k == nullptr || rest % kinds == 1;
  s.head = rest / kinds;
  // sixteens that end with the first token's unit, where there is more than one
  const int lead = p.slot && p.tokens > kv4::kUnit ? max(p.slot[0], 0) % kv4::kUnit : 0;
  s.first = (long long)block * kv4::kUnit - lead;
  return s.first < p.tokens;
}

// The cache row of token t of the list: -1 for none.
__device__ __forceinline__ int row_of(const Kv4RowsArgs& p, long long t) {
  if (t < 0 || t >= p.tokens) return -1;
  if (!p.slot) return (int)t;
  const int r = p.slot[t];
  if (r < p.cache_rows) return r;
  record_status(p.status, GDN_ERR_DEVICE_BOUNDS);
  return -1;
}

// The unit of cache row r (>= 0) for a head.
template <int D>
__device__ __forceinline__ uint8_t* unit_at(const Kv4RowsArgs& p, int r, int head) {
  const int upp_log = p.page_log - 4;   // units of a page
  const long long page = r >> p.page_log;
  return p.cache + (((page * p.h_kv + head) << upp_log) + ((r >> 4) & ((1 << upp_log) - 1))) * kv4::unit_bytes(D);
}

// A group's scale from a lane's numbers (N words of bf16 pairs), the group's lanes FROM .. TO
// apart.
template <int N, int FROM, int TO>
__device__ __forceinline__ float scale_of(const uint32_t (&w)[N]) {
  uint32_t mags = 0, tops = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    mags = max_u16x2(mags, w[i] & 0x7fff7fffu);
    tops = max_s16x2(tops, w[i]);             // (negative numbers' bits are below 0)
  }
  uint32_t ex = kv4::extremes(mags, tops);
#pragma unroll
  for (int m = FROM; m <= TO; m <<= 1) ex = max_u16x2(ex, __shfl_xor_sync(0xffffffffu, ex, m));
  return kv4::group_scale(ex);
}

__device__ __forceinline__ float lo_f32(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f32(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Codes of a group's eight channels (of lane t of four), and the group's scale: as K's word,
// or in their order, the first four and the last four a half of V's words each.
template <bool V>
__device__ __forceinline__ uint32_t codes_of(uint4 raw, float& s) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  s = scale_of<4, 1, 2>(w);
  const float r = kv4::inverse(s);
  uint32_t c = 0;                              // the highest nibble first; K: channels 7 5 3 1 6 4 2 0
#pragma unroll
  for (int k = 7; k >= 0; --k) {
    const int o = V ? k : k < 4 ? 2 * k : 2 * k - 7;
    c = c * 16 + kv4::code_bits(o % 2 ? hi_f32(w[o / 2]) : lo_f32(w[o / 2]), r);
  }
  c = s == s ? c - kv4::kCodeBase * 0x11111111u : 0x88888888u;   // of a NaN scale 8s, as of zeros
  return V ? c : __funnelshift_l(c, c, 3);
}

// Two scales as bf16, which they are exactly (a NaN keeps its bits).
__device__ __forceinline__ uint32_t scales2(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}

// Place of token j's scale of a group, from a unit's start.
template <int D>
__device__ __forceinline__ int scale_at(int j, bool is_v, int group) {
  return 16 * D + (j * (D / 16) + (is_v ? D / 32 : 0) + group) * 2;
}

// Whether the rows of V's two (at d = 64 four) tokens per lane, the warp's sixteen together,
// are one unit in order; its first row in `start`.
template <int NH>
__device__ __forceinline__ bool one_unit(const int (&row)[NH][2], int j0, int& start) {
  bool run = true;
  start = __shfl_sync(0xffffffffu, row[0][0] - j0, 0);
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int par = 0; par < 2; ++par) run = run && row[h][par] >= 0 && row[h][par] - (j0 + 8 * h + par) == start;
  return __all_sync(0xffffffffu, run) && start % kv4::kUnit == 0;
}

// Words 4 vec .. 4 vec + 3 of 16 tokens' K or V, a warp: lane 4 j + t reads channels 8 t ..
// 8 t + 7 of token j (and, at d = 64, of token j + 8) in four groups.  That is K's vector as it
// stands; V's wants two tokens' four channels, which two lanes hand over.
template <int D, bool V>
__device__ __forceinline__ void store_vector(const uint16_t* const (&src)[D == 64 ? 2 : 1], uint8_t* const (&unit)[D == 64 ? 2 : 1],
                                             const int (&row)[D == 64 ? 2 : 1], uint8_t* run, int vec) {
  constexpr int R = D / 32, NH = R == 2 ? 2 : 1, NG = 4 / NH;
  const int lane = threadIdx.x % 32, t = lane % 4, g0 = 4 * vec % R;
  uint4 raw[4];
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      raw[h * NG + i] = make_uint4(0, 0, 0, 0);
      if (src[h]) raw[h * NG + i] = __ldcs(reinterpret_cast<const uint4*>(src[h] + (g0 + i) * 32));
    }
  uint32_t c[4];
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = codes_of<V>(raw[i], s[i]);
  if (V && run) {
    const int g = lane / 4, from = 8 * t + g / 2;   // token 2 t's lane with channels 4 g .. 4 g + 3
    const uint32_t pick = g % 2 ? 0x7632 : 0x5410;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __byte_perm(__shfl_sync(0xffffffffu, c[i], from), __shfl_sync(0xffffffffu, c[i], from + 4), pick);
    *reinterpret_cast<uint4*>(run + 8 * D + 512 * vec + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
  }
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    if (!unit[h]) continue;
    const int j = row[h] % kv4::kUnit, w0 = j / 8 * R + g0;
    if constexpr (!V) {
      uint8_t* at = unit[h] + 512 * (w0 / 4) + 16 * (j % 8 * 4 + t) + w0 % 4 * 4;
      if constexpr (NG == 4) *reinterpret_cast<uint4*>(at) = make_uint4(c[0], c[1], c[2], c[3]);
      else *reinterpret_cast<uint2*>(at) = make_uint2(c[2 * h], c[2 * h + 1]);
    } else if (!run) {
      // halves j % 2 of lanes 4 g + j % 8 / 2, g = 2 t and 2 t + 1
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const int w = w0 + i;
        uint8_t* at = unit[h] + 8 * D + 512 * (w / 4) + 16 * (8 * t + j % 8 / 2) + w % 4 * 4 + j % 2 * 2;
        *reinterpret_cast<uint16_t*>(at) = (uint16_t)c[h * NG + i];
        *reinterpret_cast<uint16_t*>(at + 64) = (uint16_t)(c[h * NG + i] >> 16);
      }
    }
    if (t == 0) {
      uint8_t* at = unit[h] + scale_at<D>(j, V, g0);
      if constexpr (NG == 4) *reinterpret_cast<uint2*>(at) = make_uint2(scales2(s[0], s[1]), scales2(s[2], s[3]));
      else *reinterpret_cast<uint32_t*>(at) = scales2(s[2 * h], s[2 * h + 1]);
    }
  }
}

// A warp takes `vectors` vectors of its 16 tokens, all of a half's rows where there is work for
// every warp of the GPU even so.
template <int D>
__global__ void __launch_bounds__(kKv4Warps * 32) kv4_store_kernel(Kv4RowsArgs p, unsigned items, int vectors) {
  constexpr int NH = D == 64 ? 2 : 1, PER_HALF = D / 128 > 0 ? D / 128 : 1;   // vectors of eight tokens
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x % 32;
  const unsigned item = blockIdx.x * kKv4Warps + threadIdx.x / 32;
  Share sh;
  if (item >= items || !share_of<D>(p, item, vectors, sh)) return;
  const int j0 = D == 64 ? lane / 4 : sh.vec / PER_HALF * 8 + lane / 4;
  const uint16_t* const from = (sh.is_v ? p.v + sh.head * p.v_sh : p.k + sh.head * p.k_sh) + lane % 4 * 8;
  const long long stride = sh.is_v ? p.v_st : p.k_st;
  const uint16_t* src[NH];
  uint8_t* unit[NH];
  int row[NH];
  bool ordered = true;
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    const long long tok = sh.first + j0 + 8 * h;
    row[h] = row_of(p, tok);
    src[h] = tok >= 0 && tok < p.tokens ? from + tok * stride : nullptr;
    unit[h] = row[h] >= 0 ? unit_at<D>(p, row[h], sh.head) : nullptr;
  }
  // V's tokens one unit (half of one, above d = 64), each where its place in the list says?
  const int start = __shfl_sync(0xffffffffu, row[0] - j0, 0);
#pragma unroll
  for (int h = 0; h < NH; ++h) ordered = ordered && row[h] >= 0 && row[h] - (j0 + 8 * h) == start;
  uint8_t* run = nullptr;
  if (__all_sync(0xffffffffu, ordered) && start % kv4::kUnit == 0) run = unit[0];   // (every lane's the same)
  for (int v = sh.vec; v < sh.vec + vectors; ++v) {
    if (sh.is_v) store_vector<D, true>(src, unit, row, run, v);
    else store_vector<D, false>(src, unit, row, nullptr, v);
  }
}

// Two codes (bits 0..3 and 16..19) times a scale: code - 8 as bf16 pairs, then either the
// product rounded once to bf16 or the exact one in fp32.
__device__ __forceinline__ uint32_t less8(uint32_t x) {
  uint32_t y = (x & 0x000f000fu) | 0x43004300u;               // 128 + code
  asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(y) : "r"(0x43084308u));
  return y;
}
__device__ __forceinline__ uint32_t times(uint32_t x, uint32_t s2) {
  uint32_t y;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(s2));
  return y;
}
__device__ __forceinline__ float2 times_f32(uint32_t x, float s) {
  return make_float2(__uint_as_float(x << 16) * s, __uint_as_float(x & 0xffff0000u) * s);
}

// N pairs of one row times their scale (bf16 bits) to out + at.
template <int N, bool F32>
__device__ __forceinline__ void put(void* out, long long at, const uint32_t (&x)[N], uint32_t scale) {
  if constexpr (F32) {
    float* o = static_cast<float*>(out) + at;
    const float s = __uint_as_float(scale << 16);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 a = times_f32(x[i], s), b = times_f32(x[i + 1], s);
      *reinterpret_cast<float4*>(o + 2 * i) = make_float4(a.x, a.y, b.x, b.y);
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + at;
    const uint32_t s2 = scale | scale << 16;
    if constexpr (N == 4)
      *reinterpret_cast<uint4*>(o) = make_uint4(times(x[0], s2), times(x[1], s2), times(x[2], s2), times(x[3], s2));
    else
      *reinterpret_cast<uint2*>(o) = make_uint2(times(x[0], s2), times(x[1], s2));
  }
}

template <int D, bool F32>
__global__ void __launch_bounds__(kKv4Warps * 32) kv4_load_kernel(Kv4RowsArgs p, unsigned items) {
  constexpr int R = D / 32, NH = R == 2 ? 2 : 1, NG = 4 / NH;   // groups of a token in a vector
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x % 32;
  const unsigned item = blockIdx.x * kKv4Warps + threadIdx.x / 32;
  Share sh;
  if (item >= items || !share_of<D>(p, item, 1, sh)) return;
  const int g0 = 4 * sh.vec % R;
  if (!sh.is_v) {
    const int t = lane % 4, j0 = 4 * sh.vec / R * 8 + lane / 4;
    uint32_t word[NH][NG], sc[NH][NG / 2];
    bool there[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const int r = row_of(p, sh.first + j0 + 8 * h);
      there[h] = r >= 0;
#pragma unroll
      for (int i = 0; i < NG; ++i) word[h][i] = sc[h][i / 2] = 0;   // (a scale of zero: zeros)
      if (r < 0) continue;
      const uint8_t* u = unit_at<D>(p, r, sh.head);
      const int j = r % kv4::kUnit;
      const uint8_t* at = u + 512 * ((j / 8 * R + g0) / 4) + 16 * ((j % 8) * 4 + t) + (j / 8 * R + g0) % 4 * 4;
      if constexpr (NG == 4) {
        const uint4 w = *reinterpret_cast<const uint4*>(at);
        word[h][0] = w.x, word[h][1] = w.y, word[h][2] = w.z, word[h][3] = w.w;
        const uint2 s = *reinterpret_cast<const uint2*>(u + scale_at<D>(j, false, g0));
        sc[h][0] = s.x, sc[h][1] = s.y;
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(at);
        word[h][0] = w.x, word[h][1] = w.y;
        sc[h][0] = *reinterpret_cast<const uint32_t*>(u + scale_at<D>(j, false, 0));
      }
    }
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const long long tok = sh.first + j0 + 8 * h;
      if (tok < 0 || tok >= p.tokens) continue;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const uint32_t c = __funnelshift_r(word[h][i], word[h][i], 3), s = sc[h][i / 2] >> (16 * (i % 2)) & 0xffffu;
        uint32_t x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = there[h] ? less8(c >> (4 * k)) : 0;
        put<4, F32>(p.k_out, (tok * p.h_kv + sh.head) * D + (g0 + i) * 32 + 8 * t, x, s);
      }
    }
  } else {
    const int g = lane / 4, j0 = 4 * sh.vec / R * 8 + 2 * (lane % 4);
    int row[NH][2];
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int par = 0; par < 2; ++par) row[h][par] = row_of(p, sh.first + j0 + 8 * h + par);
    uint32_t half[4][2], sc[NH][2][NG / 2];
    int start;
    const bool run = one_unit(row, j0, start);
    if (run) {
      const uint4 w = *reinterpret_cast<const uint4*>(unit_at<D>(p, start, sh.head) + 8 * D + 512 * sh.vec + 16 * lane);
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) half[i][0] = x[i] & 0xffffu, half[i][1] = x[i] >> 16;
    }
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int par = 0; par < 2; ++par) {
        const int r = row[h][par], j = r % kv4::kUnit;
#pragma unroll
        for (int i = 0; i < NG / 2; ++i) sc[h][par][i] = 0;
        if (r < 0) continue;
        const uint8_t* u = unit_at<D>(p, r, sh.head);
        if (!run) {
          const uint16_t* at = reinterpret_cast<const uint16_t*>(u + 8 * D + 16 * (4 * g + j % 8 / 2) + 2 * (j % 2));
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const int w = j / 8 * R + (R == 2 ? i : g0 + i);
            half[NH == 2 ? 2 * h + i : i][par] = at[256 * (w / 4) + 2 * (w % 4)];
          }
        }
        if constexpr (NG == 4) {
          const uint2 s = *reinterpret_cast<const uint2*>(u + scale_at<D>(j, true, g0));
          sc[h][par][0] = s.x, sc[h][par][1] = s.y;
        } else {
          sc[h][par][0] = *reinterpret_cast<const uint32_t*>(u + scale_at<D>(j, true, 0));
        }
      }
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int par = 0; par < 2; ++par) {
        const long long tok = sh.first + j0 + 8 * h + par;
        if (tok < 0 || tok >= p.tokens) continue;
        const bool there = row[h][par] >= 0;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const uint32_t c = half[NH == 2 ? 2 * h + i : i][par], s = sc[h][par][i / 2] >> (16 * (i % 2)) & 0xffffu;
          const uint32_t d = c >> 8;           // channels 0, 1 and 2, 3: the second nibble to bit 16
          const uint32_t x[2] = {there ? less8(c | c << 12) : 0, there ? less8(d | d << 12) : 0};
          put<2, F32>(p.v_out, (tok * p.h_kv + sh.head) * D + (g0 + i) * 32 + 4 * g, x, s);
        }
      }
  }
}

template <int D>
cudaError_t launch_d(const Kv4RowsArgs& p, bool load, cudaStream_t stream, int sms) {
  const int kinds = (p.k != nullptr) + (p.v != nullptr);
  // one sixteen more than the tokens fill: the first may be part of one
  const long long blocks16 = (p.tokens + kv4::kUnit - 1) / kv4::kUnit + (p.slot && p.tokens > kv4::kUnit ? 1 : 0);
  long long items = blocks16 * p.h_kv * kinds * (D / 64);
  // d = 256 has two vectors to eight tokens' rows: a warp takes both once each SM has 32 warps
  const int vectors = !load && D == 256 && items >= 64LL * sms ? 2 : 1;
  items /= vectors;
  const long long grid = (items + kKv4Warps - 1) / kKv4Warps;
  if (grid > 0x7fffffffLL || items > 0xffffffffLL) return cudaErrorInvalidValue;
  cudaLaunchAttribute overlap;
  overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  overlap.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kKv4Warps * 32);
  cfg.stream = stream;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  if (!load) return cudaLaunchKernelEx(&cfg, kv4_store_kernel<D>, p, (unsigned)items, vectors);
  return cudaLaunchKernelEx(&cfg, p.out_f32 ? kv4_load_kernel<D, true> : kv4_load_kernel<D, false>, p, (unsigned)items);
}

cudaError_t launch_rows(const Kv4RowsArgs& p, bool load, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  switch (p.d) {
    case 64: return launch_d<64>(p, load, stream, sms);
    case 128: return launch_d<128>(p, load, stream, sms);
    case 256: return launch_d<256>(p, load, stream, sms);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_kv4_store(const Kv4RowsArgs& p, cudaStream_t stream) { return launch_rows(p, false, stream); }
cudaError_t launch_kv4_load(const Kv4RowsArgs& p, cudaStream_t stream) { return launch_rows(p, true, stream); }

}  // namespace gdn
