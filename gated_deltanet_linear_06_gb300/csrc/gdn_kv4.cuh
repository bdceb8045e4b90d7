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

// Scale of a group with the given extremes: -m / 8, m of largest magnitude, the positive
// one of two alike; exact in bf16, as m is.
__device__ __forceinline__ float group_scale(float hi, float lo, bool finite) {
  const float m = hi >= -lo ? hi : lo;
  if (!finite) return __uint_as_float(0x7fc00000u);
  return fabsf(m) < kTiny ? 0.0f : m * -0.125f;
}

// Code 0 .. 15 of x.  x / s is 8 significant bits over 8, at least 2^-17 of itself away
// from a half-integer that it does not equal, so the division's rounding moves no code.
__device__ __forceinline__ uint32_t code_of(float x, float s) {
  if (!(fabsf(s) > 0.0f)) return 8;   // zeros, and NaN scales
  return (uint32_t)(__float2int_rn(fminf(fmaxf(__fdiv_rn(x, s), -8.0f), 7.0f)) + 8);
}

}  // namespace kv4
}  // namespace gdn
