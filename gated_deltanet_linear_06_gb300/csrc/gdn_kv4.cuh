// gdn_kv4.cuh -- the 4-bit cache's format (include/gdn.h), shared by the kernels that
// write it, read it back and attend over it.
//
// A unit is 16 tokens of one kv head: 8 d bytes of K codes, 8 d of V codes, 2 d of
// bf16 scales [token][K groups | V groups].  The codes stand as the tensor cores'
// operands want them, so that attention loads whole 16-byte vectors, lane after lane,
// and needs no exchange between lanes: lane 4 g + t of mma.m16n8k16 holds, of K as the
// first operand, tokens g and g + 8 and a group's channels 8 t .. 8 t + 7; of V
// transposed as the first operand, channels 4 g .. 4 g + 3 and tokens 2 t, 2 t + 1,
// 2 t + 8, 2 t + 9.  Word w = (token / 8) * (d / 32) + group of a lane is word w % 4 of
// its vector w / 4, and vector v of lane l is at 512 v + 16 l.
#pragma once
#include <stdint.h>

#include "gdn_common.cuh"

namespace gdn {
namespace kv4 {

constexpr int kUnit = 16;    // tokens
constexpr int kGroup = 32;   // channels of one scale

__host__ __device__ constexpr int unit_bytes(int d) { return 18 * d; }

// A group whose largest magnitude is below this is held as zeros: no scale, and no
// product of a scale with a softmax weight, comes near fp32's smallest numbers.
constexpr float kTiny = 8.077935669463161e-28f;   // 2^-90

// Extremes of numbers as bf16 pairs, both as their bits: the largest magnitude in the low
// half, the largest number (0 where none is positive) in the high half.  Bits of magnitudes
// are in the numbers' order, an infinity and NaN above all.
__device__ __forceinline__ uint32_t extremes(uint32_t mags, uint32_t tops) {
  const uint32_t m = max(mags & 0xffffu, mags >> 16), t = max(tops & 0xffffu, tops >> 16);
  return m | t << 16;
}

// Scale of a group with these extremes: -m / 8, m of largest magnitude, the positive one of
// two alike; exact in bf16, as m is.
__device__ __forceinline__ float group_scale(uint32_t extremes) {
  const uint32_t mag = extremes & 0xffffu;
  if (mag >= 0x7f80u) return __uint_as_float(0x7fc00000u);
  const float m = __uint_as_float(mag << 16);
  return m < kTiny ? 0.0f : extremes >> 16 == mag ? m * -0.125f : m * 0.125f;
}

// Code of x plus kCodeBase, modulo 2^32, with r = 1 / s (a few steps off at most): x r to a
// multiple of 2^-13 (the step of numbers around 1536), then to a whole number, ties to even both.
// With significands X and M of x and of the group's extreme (8 bits each) and e >= 0 their
// exponents' distance, |x / s| = 8 X / (2^e M) is at least 1 / (2^(e+1) M) from a half-integer that
// it does not equal, and near one e <= 4 (as 8 X / (2^e M) is about 1/2 at the least): more than
// 2^-13, which half a step of 2^-13 and r's error do not bridge; and where it equals one, both
// leave it there.  No quotient is below -8.
constexpr uint32_t kCodeBase = 0x4b400000u;
__device__ __forceinline__ uint32_t code_bits(float x, float r) {
  const float q = fminf(fmaf(x, r, 1536.0f), 1536.0f + 7.0f);
  return __float_as_uint(q + (12582912.0f + 8.0f - 1536.0f));
}

// 1 / s for code_bits; of a group without a scale (zeros) one that makes every code 8.
__device__ __forceinline__ float inverse(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return s == 0.0f ? 0.0f : r;
}

}  // namespace kv4
}  // namespace gdn
