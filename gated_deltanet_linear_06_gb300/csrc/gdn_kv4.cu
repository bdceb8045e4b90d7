// gdn_kv4.cu -- rows of k and v into the 4-bit cache (gdn_kv4_store) and back out of it
// (gdn_kv4_load).
//
// Both are streams: a row is read once and written once, and what little arithmetic
// there is (a group's extremes, 32 divisions) hides under them.  The work is cut the
// way the cache's vectors lie: a warp takes 16 tokens of the list, one head, K or V and
// one 16-byte vector per lane, so each lane makes (or takes apart) whole vectors: of K
// four groups' eight channels of one token, whichever unit the token goes to; of V two
// tokens' four channels of four groups, which are one vector only where the 16 tokens
// are a unit.  Elsewhere (a decode step's rows, one of each sequence) V's pieces are two
// bytes each.  When the list runs through units it need not begin with one: the tokens
// are taken in sixteens that end where the first token's unit does.
#include "../../include/gdn.h"
#include "gdn_kv4.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

constexpr int kKv4Warps = 8;

__device__ __forceinline__ void unpack8(uint4 raw, float (&x)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// One warp's share of a call: tokens first .. first + 15 of the list (those in range),
// head, K or V, vector.
struct Share {
  long long first;
  int head, vec;
  bool is_v;
};

template <int D>
__device__ __forceinline__ bool share_of(const Kv4RowsArgs& p, long long item, Share& s) {
  constexpr int NV = D / 64;
  const int kinds = (p.k != nullptr) + (p.v != nullptr);
  const int per = p.h_kv * kinds * NV;
  const long long block = item / per;
  int rest = (int)(item - block * per);
  s.vec = rest % NV;
  rest /= NV;
  s.is_v = p.k == nullptr || rest % kinds == 1;
  s.head = rest / kinds;
  // sixteens that end with the first token's unit, where there is more than one
  const int lead = p.slot && p.tokens > kv4::kUnit ? max(p.slot[0], 0) % kv4::kUnit : 0;
  s.first = block * kv4::kUnit - lead;
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
  const int page = r / p.page, at = (r - page * p.page) / kv4::kUnit;
  return p.cache + (((long long)page * p.h_kv + head) * (p.page / kv4::kUnit) + at) * kv4::unit_bytes(D);
}

// Codes of a group's eight channels (of lane t of four) as K's word, and the group's scale.
__device__ __forceinline__ uint32_t k_word(uint4 raw, float& s) {
  float x[8], hi, lo;
  unpack8(raw, x);
  hi = lo = x[0];
  bool finite = isfinite(x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    hi = fmaxf(hi, x[i]);
    lo = fminf(lo, x[i]);
    finite = finite && isfinite(x[i]);
  }
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    finite = __shfl_xor_sync(0xffffffffu, (int)finite, m) && finite;
  }
  s = kv4::group_scale(hi, lo, finite);
  uint32_t w = 0;
#pragma unroll
  for (int o = 0; o < 8; ++o) w |= kv4::code_of(x[o], s) << (4 * (o / 2 + 4 * (o % 2)));
  return __funnelshift_l(w, w, 3);
}

// Codes of a group's four channels (of lane group g of eight) as half a word of V.
__device__ __forceinline__ uint32_t v_half(uint2 raw, float& s) {
  const float x[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u),
                      __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xffff0000u)};
  float hi = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), lo = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
  bool finite = isfinite(x[0]) && isfinite(x[1]) && isfinite(x[2]) && isfinite(x[3]);
#pragma unroll
  for (int m = 4; m <= 16; m <<= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    finite = __shfl_xor_sync(0xffffffffu, (int)finite, m) && finite;
  }
  s = kv4::group_scale(hi, lo, finite);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= kv4::code_of(x[i], s) << (4 * i);
  return w;
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

template <int D>
__global__ void __launch_bounds__(kKv4Warps * 32) kv4_store_kernel(Kv4RowsArgs p, long long items) {
  constexpr int R = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x % 32;
  const long long item = (long long)blockIdx.x * kKv4Warps + threadIdx.x / 32;
  Share sh;
  if (item >= items || !share_of<D>(p, item, sh)) return;
  if (!sh.is_v) {
    const int t = lane % 4;
    uint4 raw[4];
    int row[2] = {-1, -1};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // word 4 vec + i: of the token at w / R * 8 + lane / 4, group w % R
      const int w = 4 * sh.vec + i, j = w / R * 8 + lane / 4;
      const long long tok = sh.first + j;
      if (i == 0 || (R == 2 && i == 2)) row[i / 2] = row_of(p, tok);
      raw[i] = make_uint4(0, 0, 0, 0);
      if (row[R == 2 ? i / 2 : 0] >= 0)
        raw[i] = *reinterpret_cast<const uint4*>(p.k + tok * p.k_st + sh.head * p.k_sh + (w % R) * 32 + 8 * t);
    }
    uint32_t word[4];
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) word[i] = k_word(raw[i], s[i]);
    if constexpr (R >= 4) {
      if (row[0] < 0) return;
      uint8_t* u = unit_at<D>(p, row[0], sh.head);
      const int j = row[0] % kv4::kUnit, g0 = 4 * sh.vec % R;
      const int vec = (j / 8 * R + g0) / 4;
      *reinterpret_cast<uint4*>(u + 512 * vec + 16 * ((j % 8) * 4 + t)) =
          make_uint4(word[0], word[1], word[2], word[3]);
      if (t == 0)
        *reinterpret_cast<uint2*>(u + scale_at<D>(j, false, g0)) =
            make_uint2(scales2(s[0], s[1]), scales2(s[2], s[3]));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (row[h] < 0) continue;
        uint8_t* u = unit_at<D>(p, row[h], sh.head);
        const int j = row[h] % kv4::kUnit;
        *reinterpret_cast<uint2*>(u + 16 * ((j % 8) * 4 + t) + j / 8 * 8) = make_uint2(word[2 * h], word[2 * h + 1]);
        if (t == 0) *reinterpret_cast<uint32_t*>(u + scale_at<D>(j, false, 0)) = scales2(s[2 * h], s[2 * h + 1]);
      }
    }
  } else {
    const int g = lane / 4, t = lane % 4;
    // rows of the two tokens of each half that this vector takes from
    constexpr int NH = R == 2 ? 2 : 1;
    int row[NH][2];
    uint2 raw[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int w = 4 * sh.vec + i;
#pragma unroll
      for (int par = 0; par < 2; ++par) {
        const long long tok = sh.first + w / R * 8 + 2 * t + par;
        int& r = row[R == 2 ? i / 2 : 0][par];
        if (i == 0 || (R == 2 && i == 2)) r = row_of(p, tok);
        raw[i][par] = make_uint2(0, 0);
        if (r >= 0)
          raw[i][par] = *reinterpret_cast<const uint2*>(p.v + tok * p.v_st + sh.head * p.v_sh + (w % R) * 32 + 4 * g);
      }
    }
    uint32_t half[4][2];
    float s[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int par = 0; par < 2; ++par) half[i][par] = v_half(raw[i][par], s[i][par]);
    // a unit of its own: every token where the first one's place says
    const int w0 = 4 * sh.vec, j0 = w0 / R * 8 + 2 * t;
    bool run = true;
    int start = 0;
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int par = 0; par < 2; ++par) {
        const int at = row[h][par] - (j0 + 8 * h + par);
        if (h == 0 && par == 0) start = __shfl_sync(0xffffffffu, at, 0);
        run = run && row[h][par] >= 0 && at == start;
      }
    run = __all_sync(0xffffffffu, run) && start % kv4::kUnit == 0;
    if (run) {
      uint8_t* u = unit_at<D>(p, start, sh.head);
      *reinterpret_cast<uint4*>(u + 8 * D + 512 * sh.vec + 16 * lane) =
          make_uint4(half[0][0] | half[0][1] << 16, half[1][0] | half[1][1] << 16, half[2][0] | half[2][1] << 16,
                     half[3][0] | half[3][1] << 16);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int par = 0; par < 2; ++par) {
        const int r = row[R == 2 ? i / 2 : 0][par];
        if (r < 0) continue;
        uint8_t* u = unit_at<D>(p, r, sh.head);
        const int j = r % kv4::kUnit, grp = (4 * sh.vec + i) % R, w = j / 8 * R + grp;
        if (!run)
          *reinterpret_cast<uint16_t*>(u + 8 * D + 512 * (w / 4) + 16 * (4 * g + j % 8 / 2) + 4 * (w % 4) + 2 * (j % 2)) =
              (uint16_t)half[i][par];
        if (g == 0) *reinterpret_cast<uint16_t*>(u + scale_at<D>(j, true, grp)) = (uint16_t)(__float_as_uint(s[i][par]) >> 16);
      }
  }
}

// n values (4 or 8) to bf16 or fp32.
template <int N, bool F32>
__device__ __forceinline__ void put(void* out, long long at, const float (&x)[N]) {
  if constexpr (F32) {
    float* o = static_cast<float*>(out) + at;
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(o + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + at;
    if constexpr (N == 8)
      *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    else
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  }
}

__device__ __forceinline__ float scale_in(const uint8_t* at) {
  return bf16_to_f32(*reinterpret_cast<const uint16_t*>(at));
}

template <int D, bool F32>
__global__ void __launch_bounds__(kKv4Warps * 32) kv4_load_kernel(Kv4RowsArgs p, long long items) {
  constexpr int R = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x % 32;
  const long long item = (long long)blockIdx.x * kKv4Warps + threadIdx.x / 32;
  Share sh;
  if (item >= items || !share_of<D>(p, item, sh)) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int w0 = 4 * sh.vec + i, grp = w0 % R;
    if (!sh.is_v) {
      const int t = lane % 4;
      const long long tok = sh.first + w0 / R * 8 + lane / 4;
      if (tok < 0 || tok >= p.tokens) continue;
      const int r = row_of(p, tok);
      float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (r >= 0) {
        const uint8_t* u = unit_at<D>(p, r, sh.head);
        const int j = r % kv4::kUnit, w = j / 8 * R + grp;
        uint32_t c = *reinterpret_cast<const uint32_t*>(u + 512 * (w / 4) + 16 * ((j % 8) * 4 + t) + 4 * (w % 4));
        const float s = scale_in(u + scale_at<D>(j, false, grp));
        c = __funnelshift_r(c, c, 3);
#pragma unroll
        for (int o = 0; o < 8; ++o) x[o] = s * (float)((int)(c >> (4 * (o / 2 + 4 * (o % 2))) & 15) - 8);
      }
      put<8, F32>(p.k_out, (tok * p.h_kv + sh.head) * D + grp * 32 + 8 * t, x);
    } else {
      const int g = lane / 4;
#pragma unroll
      for (int par = 0; par < 2; ++par) {
        const long long tok = sh.first + w0 / R * 8 + 2 * (lane % 4) + par;
        if (tok < 0 || tok >= p.tokens) continue;
        const int r = row_of(p, tok);
        float x[4] = {0, 0, 0, 0};
        if (r >= 0) {
          const uint8_t* u = unit_at<D>(p, r, sh.head);
          const int j = r % kv4::kUnit, w = j / 8 * R + grp;
          const uint32_t c = *reinterpret_cast<const uint16_t*>(u + 8 * D + 512 * (w / 4) + 16 * (4 * g + j % 8 / 2) +
                                                                4 * (w % 4) + 2 * (j % 2));
          const float s = scale_in(u + scale_at<D>(j, true, grp));
#pragma unroll
          for (int i2 = 0; i2 < 4; ++i2) x[i2] = s * (float)((int)(c >> (4 * i2) & 15) - 8);
        }
        put<4, F32>(p.v_out, (tok * p.h_kv + sh.head) * D + grp * 32 + 4 * g, x);
      }
    }
  }
}

template <int D>
cudaError_t launch_d(const Kv4RowsArgs& p, bool load, cudaStream_t stream) {
  const int kinds = (p.k != nullptr) + (p.v != nullptr);
  // one sixteen more than the tokens fill: the first may be part of one
  const long long blocks16 = (p.tokens + kv4::kUnit - 1) / kv4::kUnit + (p.slot && p.tokens > kv4::kUnit ? 1 : 0);
  const long long items = blocks16 * p.h_kv * kinds * (D / 64);
  const long long grid = (items + kKv4Warps - 1) / kKv4Warps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchAttribute overlap;
  overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  overlap.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kKv4Warps * 32);
  cfg.stream = stream;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  if (!load) return cudaLaunchKernelEx(&cfg, kv4_store_kernel<D>, p, items);
  return cudaLaunchKernelEx(&cfg, p.out_f32 ? kv4_load_kernel<D, true> : kv4_load_kernel<D, false>, p, items);
}

cudaError_t launch_rows(const Kv4RowsArgs& p, bool load, cudaStream_t stream) {
  switch (p.d) {
    case 64: return launch_d<64>(p, load, stream);
    case 128: return launch_d<128>(p, load, stream);
    case 256: return launch_d<256>(p, load, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_kv4_store(const Kv4RowsArgs& p, cudaStream_t stream) { return launch_rows(p, false, stream); }
cudaError_t launch_kv4_load(const Kv4RowsArgs& p, cudaStream_t stream) { return launch_rows(p, true, stream); }

}  // namespace gdn
