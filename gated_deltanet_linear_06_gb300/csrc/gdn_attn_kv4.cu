// gdn_attn_kv4.cu -- attention of a batch of sequences over the 4-bit paged cache
// (mma.sync tensor-core products that take the codes as they are stored).
//
// Mathematics.  A row r = (step, query head) of a sequence wants o = sum_j w_j v_j / sum_j w_j,
// w_j = 2^(s_j - ref), s_j = scale log2(e) q.k_j, for any ref.  With k_jc = a_jg c_jc, codes c and a
// scale a per token and group g of 32 channels,
//   s_j = sum_g a_jg (sum_{c in g} c_jc q_c),   o_c = sum_j c_jc (w_j b_jg),
// so the codes are multiplied as whole numbers, K's scales meet the products' sums in fp32
// and V's meet the weights before their one rounding, to fp16.
//
// What bounds it.  4.5 bits a value: at the memory's rate an SM gets 38 values a clock, and
// what it can do for each of them decides.  Taking a nibble out costs an instruction for two
// values whatever one does; so everything else is kept from costing any:
//   - the codes lie as the operands' fragments do, so a lane's words come by 16-byte loads and no
//     lane hands anything to another;
//   - four bits masked out of a word are an fp16 number already (see kAt3 below): no
//     conversion, no offset to subtract, at most one shift for two masks (those to the left
//     go to the fp32 pipe; those to the right cost 4 % more there, as products' upper halves);
//   - the 8 by which the stored codes are too large is taken off by the tensor cores: for K as
//     the value that the sum starts from, for V by a product with a constant (taking it off the
//     values was eight instructions for every one of those);
//   - up to 8 rows (a group's query heads, or several steps' of them) are the products' N, tokens
//     or channels their M, so few rows waste nothing; 9 to 16 are their M, and the scores' sums
//     are the next products' operand as they stand.
// tcgen05 takes its operands from shared memory, where each value would have to be written as
// 16 bits first, four times what is read: more than the 128 bytes a clock there.  Scales per
// (token, group) bar its 4-bit kinds, whose scales run along the other dimension for V.
// (fp8 products would need half the masks, but mma.sync's are converted to fp16 here: 40 clocks
// a product with fresh operands where fp16's takes 13.)
//
// Split.  A job is a (sequence, kv head, 8 or 16 rows).  All jobs' stages (64 tokens of d = 64 or
// 128, 32 of 256) are laid end to end, with something for each job's fixed cost, and every warp
// of a grid of one CTA an SM takes an equal share: one long sequence fills the GPU as well as
// many short ones do.  Warps share nothing but the sums of the lengths at the start; each has
// its own ring of two stages, filled by bulk copies (a page's units of a head are contiguous)
// while the other is met.  A share ends where it ends; a second launch joins a job's shares.
// Shares follow from the lengths alone and are found on the device, so a captured call stays valid
// while the lengths grow.  Only how many lane groups join a row goes by what the host knows, the
// table's width: equal calls add in equal order, those of a wider table may join in another.
//
// Softmax.  ref moves only when a score passes it by kGrow binary orders; else a stage costs a
// vote.  Weights times scales of V have to fit fp16, so weights carry a factor 2^-v that suits the
// scales, those of all groups and tokens of a stage alike, whoever sees them: that they lie near
// 2^v (13 binary orders, see kNarrow) is looked at in every stage, two instructions for two
// scales.  Where they do not, what is summed goes to the share's slot in memory, in fp32 and free
// of v, v moves, and scales that still do not fit go by themselves, those near each other at a
// time: so no scale, seen or not, takes another's bits.  64 sequences of 6001 (32, 8, 128, caches
// cold) take 98 us; 107 with half of the groups zeros, 100 with every first token's scales 2^-14
// of the others', 182 with those of one token in a hundred, 246 with half of the groups'.
//
// Measured, both launches, of the bytes that the cache holds for the tokens: 256 sequences of 100
// to 8000 tokens (16 query heads, 2 kv heads, d = 256) 119 us, 5.0 TB/s; one of 131072 (32, 8,
// 128) 38 us, 4.0 TB/s; 64 of 6001 (32, 8, 128) 86 us, 5.2 TB/s, in pages of 16 90 us; 96 of 1 to
// 2900 (64, 8, 64) 28 us, 2.9 TB/s; 17 of 4 to 6001 with 4 steps (32, 8, 128, pages of 16) 32 us,
// 1.9 TB/s; one of 833 8.5 us, latency (the lengths 0.8, first copy asked for 1.3, its rows and
// the data 1, a stage 1.4, the share written 0.5, join 2).  Per unit of 16 tokens at d = 256, of
// the full batch: 275 clocks of an SM where the memory's rate gives 217, for 538 instructions (248
// of the integer pipe, which starts one every other clock and scheduler: 124) and 40 products
// (80).  Rows above 16 of a kv head meet the same tokens in a job of their own: 64 sequences of
// 6001 with 1, 2, 4 and 8 steps (16, 2, 256: 8 to 64 rows; caches cold) 61, 104, 180 and 332 us.
// Masks, products and the fp32 arithmetic between them contend for the same issue slots and
// registers' ports, and their times add up: 12 warps with stages of half the size took 132 us for
// 114, the next stage's scores between a stage's sums 133, stages of 3 units (registers run out)
// 129.
#include <limits.h>
#include <math.h>

#include "../../include/gdn.h"
#include "gdn_attn_ranges.h"
#include "gdn_kv4.cuh"
#include "gdn_launch.h"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr long long kWaitClocks = 2000000000LL;   // a second or so: a copy that has not come by then never will
// A row's weights are 2^(score - ref); where ref moves the largest comes to 2^(kTop - v), a power of
// two, so that its products with scales are exact in fp16 (with ref a whole number one output in ten
// was not the exact one rounded, with this one in thirteen).  Scores may then grow by kGrow binary orders, and V's scales lie from
// 2^(v - kNarrow) to 2^(v + kWide): a weight times a scale stays below 2^15, in fp16, and what
// fp16's subnormal numbers round off, 2^-25 at most next to 2^(kTop - kNarrow), is 2^-23 of the
// row's largest weight times the least scale there is.
constexpr float kTop = 8.0f, kGrow = 4.0f;
constexpr int kWide = 3, kNarrow = 10;
constexpr int kLeastV = -93;                       // scales are zero or at least 2^-93
constexpr int kMostV = 60;                         // with a larger v, weights that count would be subnormal
constexpr int kStored = 28;                        // sums are held with weights of 2^(kTop + kGrow - kStored) at the most
constexpr int kMaxCtas = 160;                      // the workspace has room for
constexpr int kMaxWarps = 16;

// What both launches know of a call.
struct Kv4Plan {
  int G, R;                  // query heads of a kv head, rows of a job
  int blocks;                // blocks of rows per kv head: a job each
  int jobs_per_seq;          // h_kv * blocks
  int workers;               // warps
};

struct Kv4Params {
  AttnKv4Args a;
  Kv4Plan pl;
  float qscale;              // scale * log2(e)
  int2* span;                // per job: the first and the last worker with a share of it
  float2* ml;                // per slot and row: (reference, sum)
  float* part;               // per slot and row: d sums
};

template <int D, int NT>
struct Cfg {
  static constexpr int R = D / 32;
  static constexpr int UNITS = NT == 2 ? 256 / D : 512 / D < 4 ? 512 / D : 4;   // met at once: a stage
  // What a job costs besides its units (its rows in and out), in stages, some 640 / D units: 96
  // sequences of up to 2900 tokens of d = 64 took 40 us with 2 units, 34 with 4 and 28 with 8;
  // 256 of up to 8000 of d = 256 took 126 with 8 and 122.5 with 2.
  static constexpr int JOB = 640 / D > UNITS ? 640 / D / UNITS : 1;
  static constexpr bool QREG = NT * R <= 8;          // q's operands in registers, else in shared memory
  static constexpr bool BREG = R <= 2;               // and the sums of their channels
  static constexpr int WARPS = D == 64 && NT == 1 ? 12 : 8;   // (registers for 8 or 12; 10 left one scheduler with more)
  static constexpr int UNIT = kv4::unit_bytes(D), STAGE = UNITS * UNIT;
  static constexpr int STAGES = D == 256 && NT == 2 ? 3 : 2;
  static constexpr int WORDS = UNITS * R / 4;        // a lane's share of the words of a stage's scales of V,
  static constexpr int RUN = WORDS < R / 2 ? WORDS : R / 2;   // so many of a token's in a row
  static constexpr int QBYTES = QREG ? 0 : NT * R * 512, BBYTES = BREG ? 0 : R * 64, SBYTES = WORDS * 128;   // a warp's
  static constexpr int SMEM = WARPS * (STAGES * STAGE + QBYTES + BBYTES + SBYTES);
  static_assert(SMEM <= 216 * 1024 && UNITS * STAGES <= 32, "shared memory, bits of `bad`");
};

__device__ __forceinline__ float ex2(float x) {   // results below 2^-126: zero
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// d = a b + c over fp16, fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                    float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  mma(d, a, b0, b1, d[0], d[1], d[2], d[3]);
}

__device__ __forceinline__ float lo_f32(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f32(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Codes as fp16 values, two in a word: four bits anywhere among the lowest eleven, under zeros,
// are that code times 2^(place - 24), exactly (a subnormal number, which the tensor cores take
// as it is, or one of the least exponent, whose steps are the same).  The other operand or the
// end result makes up for the power of two, and a product takes off the 8 that each code is
// too much.  The places are the highest two there are: a product's terms are cut off below
// 2^-25 of the largest, and for a subnormal number that goes by 2^-14, whatever it is.  At places
// 0 and 4, which would spare V's words a shift, small sums next to a large weight lost what is
// below 2^-14 of it.  (K's words lie so that one shift is enough.)
constexpr uint32_t kAt3 = 0x00780078u, kAt7 = 0x07800780u;
constexpr uint32_t kLess8At3 = 0x80408040u, kLess8At7 = 0x84008400u;   // -8 at those places
constexpr int kUnit3 = -21, kUnit7 = -17;                               // what 1 is there, a power of two
constexpr uint32_t kOnes = 0x3c003c00u;

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // (-126 .. 127)
// 2^e as the bits of a bf16 number, of an exponent above -127.
__device__ __forceinline__ uint32_t bf16_pow2(int e) { return (uint32_t)(e + 127) << 7; }
// The least e with a bf16 magnitude of these bits below 2^e.
__device__ __forceinline__ int above(uint32_t m) { return (int)(m >> 7) - 126; }

// A bf16 pair times a power of two (exact) as fp16.
__device__ __forceinline__ uint32_t half_pair(uint32_t x, uint32_t up) {
  uint32_t y;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(up));
  return pack_f16x2(lo_f32(y), hi_f32(y));
}

__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred P1;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 P1, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, P1;\n\t}\n"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// W words (a multiple of 2) from shared memory, in the widest loads.
template <int W>
__device__ __forceinline__ void words_at(uint32_t (&w)[W], const uint8_t* p) {
  if constexpr (W % 4 == 0) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(p + 4 * i);
      w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
    }
  } else if constexpr (W == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x, w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

template <int D>
constexpr int kSet = D / 32 < 4 ? D / 32 : 4;   // groups whose words come together

// A lane's words of K's or V's codes of a unit: of both halves of its tokens, for a set of groups.
template <int D>
__device__ __forceinline__ void codes_at(uint32_t (&w0)[kSet<D>], uint32_t (&w1)[kSet<D>], const uint8_t* p, int lane,
                                         int set) {
  constexpr int NV = D / 64;
  const uint4* v = reinterpret_cast<const uint4*>(p) + lane;
  if constexpr (NV == 1) {
    const uint4 x = v[0];
    w0[0] = x.x, w0[1] = x.y, w1[0] = x.z, w1[1] = x.w;
  } else {
    const uint4 x = v[set * 32], y = v[(set + NV / 2) * 32];
    w0[0] = x.x, w0[1] = x.y, w0[2] = x.z, w0[3] = x.w;
    w1[0] = y.x, w1[1] = y.y, w1[2] = y.z, w1[3] = y.w;
  }
}


// Units of sequence b; a length out of range counts as none.
__device__ __forceinline__ int units_of(const AttnKv4Args& a, int b) {
  const int n = a.len[b];
  return n > 0 && n <= (long long)a.width * a.page ? (n + kv4::kUnit - 1) / kv4::kUnit : 0;
}

// What a job of n units costs, in stages of `units`: `job` for its rows in and out.
__device__ __forceinline__ int cost_of(int n, int units, int job) { return n > 0 ? (n + units - 1) / units + job : 0; }

// before[0 .. batch]: costs of a job of each sequence before, in shared memory, by the whole CTA.
template <int UNITS, int JOB>
__device__ void sum_costs(const AttnKv4Args& a, long long* before, long long* warp_sums, bool report) {
  const int threads = blockDim.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int per = (a.batch + threads - 1) / threads, b0 = threadIdx.x * per;
  long long mine = 0;
  for (int i = 0; i < per; ++i)
    if (b0 + i < a.batch) {
      const int n = a.len[b0 + i];
      if (report && (n < 0 || n > (long long)a.width * a.page)) record_status(a.status, GDN_ERR_DEVICE_BOUNDS);
      mine += cost_of(units_of(a, b0 + i), UNITS, JOB);
    }
  long long sum = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, sum, m);
    if (lane >= m) sum += o;
  }
  if (lane == 31) warp_sums[warp] = sum;
  __syncthreads();
  long long at = sum - mine;
  for (int w = 0; w < warp; ++w) at += warp_sums[w];
  for (int i = 0; i < per; ++i)
    if (b0 + i < a.batch) {
      before[b0 + i] = at;
      at += cost_of(units_of(a, b0 + i), UNITS, JOB);
      if (b0 + i == a.batch - 1) before[a.batch] = at;
    }
  __syncthreads();
}

// A warp's place among the items: what a job costs besides, then its stages, job after job.
struct Item {
  int b, job, s, n;          // sequence, job of it, stage (below 0: before the first), stages
};

// The next job's start, given the items (from the end of this job on) that are left to the
// warp; a job whose stages begin past them is none.
template <int JOB>
__device__ __forceinline__ void next_job(const Kv4Params& p, const long long* before, Item& it, long long& rest) {
  it.s = 0;
  rest -= JOB;
  if (++it.job < p.pl.jobs_per_seq) return;
  it.job = 0;
  do {
    ++it.b;
    it.n = it.b < p.a.batch ? (int)(before[it.b + 1] - before[it.b]) - JOB : 0;
  } while (it.n < 0 && it.b < p.a.batch);
}

// Which of a lane's two rows element e of its products is, and which token of a unit (of half x).
template <int NT>
__device__ __forceinline__ constexpr int row_of(int e) { return NT == 2 ? e / 2 : e % 2; }
template <int NT>
__device__ __forceinline__ int token_of(int lane, int x, int e) {
  return NT == 2 ? 8 * x + 2 * (lane % 4) + e % 2 : lane / 4 + e / 2 * 8;
}
template <int NT>
constexpr int kTokens = NT == 2 ? 4 : 2;   // of a unit that a lane has
// The scales of a lane's i-th token of unit k of a stage, K's.
template <int D, int NT>
__device__ __forceinline__ uint8_t* scales_of(uint8_t* st, int lane, int k, int i) {
  return st + k * Cfg<D, NT>::UNIT + 16 * D + (NT == 2 ? 2 * (lane % 4) + i % 2 + i / 2 * 8 : lane / 4 + 8 * i) * (D / 8);
}
// A lane's i-th run of words of a stage's scales of V, RUN words of a token's groups.
template <int D, int NT>
__device__ __forceinline__ uint32_t* v_scales(uint8_t* st, int lane, int i) {
  using C = Cfg<D, NT>;
  constexpr int RUNS = C::R / 2 / C::RUN;    // of a token
  const int x = lane + 32 * i, token = x / RUNS;
  return reinterpret_cast<uint32_t*>(st + token / kv4::kUnit * C::UNIT + 16 * D + token % kv4::kUnit * (D / 8) + D / 16 +
                                     x % RUNS * (C::RUN * 4));
}

// What a warp has summed of a job.
template <int D, int NT>
struct Sums {
  float o[D / 32][2 * NT][4];   // weights times values, in the codes' units
  float ref[2], sum[2];         // of weights times 2^(v - kStored): whatever v is
  int v;
  uint32_t fresh;               // this lane's rows that have not seen a score
  bool stands;                  // a part of the outputs' sums is in the share's slot
};

// The power of two that a stage's scales of V are to be taken relative to, given what it was: the
// largest is below it, unless they all lie near 2^v as it is.  apart: some are too small for that,
// or all too large for any; top: above the largest.
template <int D, int NT>
__device__ __forceinline__ int range_of(uint8_t* st, int lane, int v, bool& apart, int& top) {
  using C = Cfg<D, NT>;
  uint32_t most = 0, least = 0x7f80u;        // of those that are finite
#pragma unroll 1
  for (int i = 0; i < C::WORDS; ++i) {
    const uint32_t w = v_scales<D, NT>(st, lane, i / C::RUN)[i % C::RUN];
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
      const uint32_t m = w >> h & 0x7fffu;
      if (m < 0x7f80u && m >= bf16_pow2(kLeastV - kNarrow)) most = max(most, m), least = min(least, m);
    }
  }
  most = __reduce_max_sync(0xffffffffu, most);
  least = __reduce_min_sync(0xffffffffu, least);
  apart = false;
  if (most == 0) return v;
  top = above(most);
  if (most >= bf16_pow2(v + kWide) || least < bf16_pow2(v - kNarrow)) v = min(max(top, kLeastV), kMostV);
  apart = least < bf16_pow2(v - kNarrow) || top > v + kWide;
  return v;
}

// Moves the rows' references, to the largest of the scores s and to scales relative to 2^v1.
template <int D, int NT>
__device__ __forceinline__ void move_refs(Sums<D, NT>& m, float (&s)[Cfg<D, NT>::UNITS][NT][4], int v1) {
  constexpr int NU = Cfg<D, NT>::UNITS;
  constexpr int LANES_0 = NT == 2 ? 1 : 4, LANES_1 = NT == 2 ? 2 : 16;   // lane bits that tell tokens, not rows, apart
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float most = -INFINITY;                  // largest score, less ref
#pragma unroll
    for (int k = 0; k < NU; ++k)
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (row_of<NT>(e) == i) most = fmaxf(most, s[k][x][e]);
#pragma unroll
    for (int k = LANES_0; k <= LANES_1; k <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, k));
    const bool first = m.fresh >> i & 1;
    if (first && most == -INFINITY) continue;
    if (!first) most = fmaxf(most, kTop - (float)m.v);
    m.fresh &= ~(1u << i);
    const float to = m.ref[i] + (most - (kTop - (float)v1)), by = to - m.ref[i];   // (as rounded)
    m.ref[i] = to;
#pragma unroll
    for (int k = 0; k < NU; ++k)
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (row_of<NT>(e) == i) s[k][x][e] -= by;
    if (!first && by != (float)(v1 - m.v)) {
      const float f = ex2((float)(v1 - m.v) - by);
      m.sum[i] *= f;
#pragma unroll
      for (int r = 0; r < D / 32; ++r)
#pragma unroll
        for (int x = 0; x < 2 * NT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (row_of<NT>(e) == i) m.o[r][x][e] *= f;
    }
  }
  m.v = v1;
}

// Weights s of a stage to the sums.
template <int D, int NT>
__device__ __forceinline__ void add_weights(Sums<D, NT>& m, const float (&s)[Cfg<D, NT>::UNITS][NT][4]) {
  float here[2] = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < Cfg<D, NT>::UNITS; ++k)
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) here[row_of<NT>(e)] += s[k][x][e];
#pragma unroll
  for (int i = 0; i < 2; ++i) m.sum[i] = fmaf(here[i], pow2(m.v - kStored), m.sum[i]);
}

// Weights s times a stage's values to the outputs, over the 16 tokens of each unit: a pair of
// units' 8s first, a sum for all of a group's channels, then their codes.
template <int D, int NT>
__device__ __forceinline__ void add_values(Sums<D, NT>& m, const float (&s)[Cfg<D, NT>::UNITS][NT][4], uint8_t* st, int lane) {
  constexpr int NU = Cfg<D, NT>::UNITS, R = D / 32, SET = kSet<D>, TOKS = kTokens<NT>;
  constexpr bool WIDE = NT == 2;
  constexpr int PAIR = NU < 2 ? NU : 2;
  const uint32_t ones[4] = {kOnes, kOnes, kOnes, kOnes};
#pragma unroll
  for (int k0 = 0; k0 < NU; k0 += PAIR) {
    uint32_t vs[PAIR][TOKS][R / 2];
#pragma unroll
    for (int k = 0; k < PAIR; ++k)
#pragma unroll
      for (int i = 0; i < TOKS; ++i) words_at<R / 2>(vs[k][i], scales_of<D, NT>(st, lane, k0 + k, i) + D / 16);
#pragma unroll
    for (int set = 0; set < R / SET; ++set) {
      uint32_t w0[PAIR][SET], w1[PAIR][SET];
#pragma unroll
      for (int k = 0; k < PAIR; ++k) codes_at<D>(w0[k], w1[k], st + (k0 + k) * Cfg<D, NT>::UNIT + 8 * D, lane, set);
#pragma unroll
      for (int rr = 0; rr < SET; ++rr) {
        const int r = set * SET + rr;
        uint32_t w[PAIR][2 * NT];      // weights times scales, as an operand
        float off[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < PAIR; ++k) {
          float sc[TOKS];
#pragma unroll
          for (int i = 0; i < TOKS; ++i) sc[i] = r % 2 ? hi_f32(vs[k][i][r / 2]) : lo_f32(vs[k][i][r / 2]);
          const auto& y = s[k0 + k];
          if constexpr (WIDE) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                w[k][2 * x + i] = pack_f16x2(y[x][2 * i] * sc[2 * x], y[x][2 * i + 1] * sc[2 * x + 1]);
            mma(off, w[k], kOnes, kOnes);
          } else {
            w[k][0] = transpose8(pack_f16x2(y[0][0] * sc[0], y[0][1] * sc[0]));
            w[k][1] = transpose8(pack_f16x2(y[0][2] * sc[1], y[0][3] * sc[1]));
            mma(off, ones, w[k][0], w[k][1]);
          }
        }
#pragma unroll
        for (int x = 0; x < 2 * NT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m.o[r][x][e] = fmaf(off[e], -8.0f * pow2((WIDE ? x % 2 : e / 2) ? kUnit7 : kUnit3), m.o[r][x][e]);
#pragma unroll
        for (int k = 0; k < PAIR; ++k) {
          const uint32_t x0 = w0[k][rr] << 3, y0 = w1[k][rr] << 3, x1 = w0[k][rr] >> 5, y1 = w1[k][rr] >> 5;
          if constexpr (WIDE) {        // rows by channels
            mma(m.o[r][0], w[k], x0 & kAt3, y0 & kAt3);
            mma(m.o[r][1], w[k], x0 & kAt7, y0 & kAt7);
            mma(m.o[r][2], w[k], x1 & kAt3, y1 & kAt3);
            mma(m.o[r][3], w[k], x1 & kAt7, y1 & kAt7);
          } else {                     // channels by rows
            const uint32_t f0[4] = {x0 & kAt3, x0 & kAt7, y0 & kAt3, y0 & kAt7};
            const uint32_t f1[4] = {x1 & kAt3, x1 & kAt7, y1 & kAt3, y1 & kAt7};
            mma(m.o[r][0], f0, w[k][0], w[k][1]);
            mma(m.o[r][1], f1, w[k][0], w[k][1]);
          }
        }
      }
    }
  }
}

// The outputs' sums, with weights that carry 2^-vo, to the share's slot, on top of what stands
// there; the weights' too.
template <int D, int NT>
__device__ __forceinline__ void put_sums(const Sums<D, NT>& m, int vo, float* part, float2* ml, int lane) {
  constexpr bool WIDE = NT == 2;
  constexpr int LANES_0 = WIDE ? 1 : 4, LANES_1 = WIDE ? 2 : 16;
  const int g = lane / 4, t = lane % 4;
  const float at3 = pow2(vo - kStored - kUnit3), at7 = pow2(vo - kStored - kUnit7);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float l = m.sum[i];
#pragma unroll
    for (int k = LANES_0; k <= LANES_1; k <<= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
    const int row = WIDE ? 8 * i + g : 2 * t + i;
    const float to = m.ref[i] - (float)(m.v - kStored);
    float keep = 0.0f;                       // (references never move down)
    if (m.stands) keep = ex2(fminf(ml[row].x - to, 0.0f));
    __syncwarp();
    if ((WIDE ? t : g) == 0) ml[row] = make_float2(to, l);
#pragma unroll
    for (int r = 0; r < D / 32; ++r)
#pragma unroll
      for (int e = i; e < (WIDE ? i + 2 : i + 1); ++e) {
        const int c = WIDE ? i + e : i;      // element of a row's channels 8 t + 4 (e - i) + 0 .. 3 or 4 g + 0 .. 3
        float4* const at = reinterpret_cast<float4*>(part + row * D + 32 * r + (WIDE ? 8 * t + 4 * (e - i) : 4 * g));
        float4 x;
        if constexpr (WIDE) x = make_float4(m.o[r][0][c] * at3, m.o[r][1][c] * at7, m.o[r][2][c] * at3, m.o[r][3][c] * at7);
        else x = make_float4(m.o[r][0][c] * at3, m.o[r][0][2 + c] * at7, m.o[r][1][c] * at3, m.o[r][1][2 + c] * at7);
        if (m.stands) {
          const float4 y = *at;
          x = make_float4(fmaf(y.x, keep, x.x), fmaf(y.y, keep, x.y), fmaf(y.z, keep, x.z), fmaf(y.w, keep, x.w));
        }
        *at = x;
      }
  }
  __syncwarp();
}

// Of a stage whose scales of V do not fit next to each other: leaves those in [lo, hi) (bits of
// magnitudes), times 2^up, and those that are not finite, the others zeros; what the stage held
// stands aside from the first time (save).  Returns the largest below lo.
template <int D, int NT>
__device__ __forceinline__ uint32_t leave(uint8_t* st, uint32_t* aside, int lane, uint32_t lo, uint32_t hi, int up, bool save) {
  using C = Cfg<D, NT>;
  uint32_t below = 0;
  __syncwarp();
#pragma unroll 1
  for (int i = 0; i < C::WORDS; ++i) {
    uint32_t* const at = v_scales<D, NT>(st, lane, i / C::RUN) + i % C::RUN;
    if (save) aside[32 * i + lane] = *at;
    const uint32_t w = aside[32 * i + lane];
    uint32_t x = 0;
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
      const uint32_t b = w >> h & 0xffffu, m = b & 0x7fffu;
      if (m >= 0x7f80u) x |= b << h;
      else if (m >= lo && m < hi) x |= (b + ((uint32_t)up << 7)) << h;
      else if (m < lo && m >= bf16_pow2(kLeastV - kNarrow)) below = max(below, m);
    }
    *at = x;
  }
  __syncwarp();
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the stage's next copy
  return __reduce_max_sync(0xffffffffu, below);
}

// Weights s times what stands of a stage's values, relative to 2^top, to the share's slot.
template <int D, int NT>
__device__ __forceinline__ void add_to_slot(const float (&s)[Cfg<D, NT>::UNITS][NT][4], uint8_t* st, int top, float* part,
                                            int lane) {
  constexpr int R = D / 32, TOKS = kTokens<NT>;
  constexpr bool WIDE = NT == 2;
  const int g = lane / 4, t = lane % 4;
  const float at3 = pow2(top - kStored - kUnit3), at7 = pow2(top - kStored - kUnit7);
  const uint32_t ones[4] = {kOnes, kOnes, kOnes, kOnes};
#pragma unroll 1
  for (int r = 0; r < R; ++r) {
    float o[2 * NT][4], off[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int x = 0; x < 2 * NT; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[x][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < Cfg<D, NT>::UNITS; ++k) {
      const uint8_t* const codes = st + k * Cfg<D, NT>::UNIT + 8 * D + 16 * lane;
      const uint32_t w0 = *reinterpret_cast<const uint32_t*>(codes + 512 * (r / 4) + r % 4 * 4);
      const uint32_t w1 = *reinterpret_cast<const uint32_t*>(codes + 512 * ((R + r) / 4) + (R + r) % 4 * 4);
      const uint32_t x0 = w0 << 3, y0 = w1 << 3, x1 = w0 >> 5, y1 = w1 >> 5;
      float sc[TOKS];
#pragma unroll
      for (int i = 0; i < TOKS; ++i)
        sc[i] = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(scales_of<D, NT>(st, lane, k, i) + D / 16)[r] << 16);
      const auto& y = s[k];
      if constexpr (WIDE) {
        uint32_t w[4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            w[2 * x + i] = pack_f16x2(y[x][2 * i] * sc[2 * x], y[x][2 * i + 1] * sc[2 * x + 1]);
        mma(off, w, kOnes, kOnes);
        mma(o[0], w, x0 & kAt3, y0 & kAt3);
        mma(o[1], w, x0 & kAt7, y0 & kAt7);
        mma(o[2], w, x1 & kAt3, y1 & kAt3);
        mma(o[3], w, x1 & kAt7, y1 & kAt7);
      } else {
        const uint32_t b0 = transpose8(pack_f16x2(y[0][0] * sc[0], y[0][1] * sc[0]));
        const uint32_t b1 = transpose8(pack_f16x2(y[0][2] * sc[1], y[0][3] * sc[1]));
        const uint32_t f0[4] = {x0 & kAt3, x0 & kAt7, y0 & kAt3, y0 & kAt7}, f1[4] = {x1 & kAt3, x1 & kAt7, y1 & kAt3, y1 & kAt7};
        mma(off, ones, b0, b1);
        mma(o[0], f0, b0, b1);
        mma(o[1], f1, b0, b1);
      }
    }
#pragma unroll
    for (int x = 0; x < 2 * NT; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool hi = WIDE ? x % 2 : e / 2;
        o[x][e] = fmaf(off[e], -8.0f * pow2(hi ? kUnit7 : kUnit3), o[x][e]) * (hi ? at7 : at3);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < NT; ++k) {         // four channels of this lane's row i, of each half
        const int row = WIDE ? 8 * i + g : 2 * t + i, c = WIDE ? 2 * i + k : i;
        float4* const at = reinterpret_cast<float4*>(part + row * D + 32 * r + (WIDE ? 8 * t + 4 * k : 4 * g));
        float4 y = *at;
        if constexpr (WIDE) y.x += o[0][c], y.y += o[1][c], y.z += o[2][c], y.w += o[3][c];
        else y.x += o[0][c], y.y += o[0][2 + c], y.z += o[1][c], y.w += o[1][2 + c];
        *at = y;
      }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::WARPS * 32, 1) attn_kv4_kernel(Kv4Params p) {
  using C = Cfg<D, NT>;
  constexpr int R = C::R;                    // groups
  constexpr bool QREG = C::QREG, BREG = C::BREG;
  // 8 rows are the products' N: a lane has tokens g, g + 8 of a unit and rows 2 t, 2 t + 1 (element
  // e of a product: token g + 8 (e / 2), row 2 t + e % 2).  16 are their M: it has tokens 2 t,
  // 2 t + 1 (of half x) and rows g, g + 8 (e / 2), the weights come out as the next products
  // want them, and the 8s of all of a group's channels take one product instead of two for
  // every 8 rows.
  constexpr bool WIDE = NT == 2;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ long long before[GDN_ATTN_MAX_BATCH + 1];
  __shared__ long long warp_sums[kMaxWarps];
  __shared__ uint64_t full[C::WARPS * C::STAGES];
  const AttnKv4Args& a = p.a;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, t = lane % 4;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  uint64_t* bar = full + warp * C::STAGES;
  if (lane == 0)
    for (int i = 0; i < C::STAGES; ++i) tc::mbar_init(bar + i, 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  sum_costs<C::UNITS, C::JOB>(a, before, warp_sums, blockIdx.x == 0);

  // This warp's items, and where the first one is.
  const long long total = before[a.batch] * p.pl.jobs_per_seq;
  const int worker = warp * gridDim.x + blockIdx.x;   // few workers: on many SMs
  const int workers = total < p.pl.workers ? (int)total : p.pl.workers;   // (none without an item)
  const long long x0 = worker < workers ? total * worker / workers : 0;
  const long long x1 = worker < workers ? total * (worker + 1) / workers : 0;
  bool ok = true;
  if (x0 < x1) {
    Item use;
    {
      int lo = 0, hi = a.batch;              // the last sequence that begins at or before x0
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (before[mid] * p.pl.jobs_per_seq <= x0) lo = mid; else hi = mid;
      }
      use.b = lo;
      const int cost = (int)(before[lo + 1] - before[lo]);
      const long long at = x0 - before[lo] * p.pl.jobs_per_seq;
      use.n = cost - C::JOB;
      use.job = (int)(at / cost);
      use.s = (int)(at - (long long)use.job * cost) - C::JOB;
    }
    long long rest = x1 - x0;                // stages not yet met
    if (use.s < 0) {                         // the share begins before the job's first stage
      rest += use.s;
      use.s = 0;
    }
    Item ask = use;
    long long to_ask = rest;                 // stages not yet asked for
    int ask_len = units_of(a, ask.b), ask_u = ask.s * C::UNITS;   // the sequence's units, the next one
    const int upp_log = 31 - __clz(a.page / kv4::kUnit);   // units of a page
    const long long page_bytes = (long long)a.h_kv * C::UNIT << upp_log;
    int entry = 0, entry_0 = INT_MIN;        // this lane's of 32 entries of the sequence's table
    const auto head_of = [&]() { return a.cache + ((long long)(ask.job / p.pl.blocks) * C::UNIT << upp_log); };
    const uint8_t* head = head_of();         // page 0's units of the job's head
    uint32_t bad = 0;                        // units of the stages whose page there is not
    const uint32_t stages = tc::smem_u32(ring) + warp * C::STAGES * C::STAGE;
    int put = 0, get = 0;
    uint32_t parity = 0;

    // One more stage: a lane for each unit, or where a page holds a whole stage one for all.
    const auto request = [&]() {
      const int units = min(C::UNITS, ask_len - ask_u);
      const int page_0 = ask_u >> upp_log, mine = ask_u + lane;
      if (page_0 < entry_0 || page_0 + C::UNITS > entry_0 + 32) {
        entry_0 = page_0;
        entry = page_0 + lane < a.width ? a.table[(long long)ask.b * a.width + page_0 + lane] : -1;
      }
      const int page = __shfl_sync(0xffffffffu, entry, (mine >> upp_log) - entry_0);
      const bool there = (unsigned)page < (unsigned)a.n_pages;
      if (lane < units && !there) record_status(a.status, GDN_ERR_DEVICE_BOUNDS);
      const uint32_t found = __ballot_sync(0xffffffffu, lane < units && there);
      const bool whole = 1 << upp_log >= C::UNITS;
      bad &= ~(((1u << C::UNITS) - 1) << (put * C::UNITS));
      bad |= (((1u << units) - 1) & ~found) << (put * C::UNITS);
      const uint32_t b = tc::smem_u32(bar + put);
      if (lane == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(b), "r"(__popc(found) * C::UNIT)
                     : "memory");
      if (lane < units && there && (!whole || lane == 0)) {
        const uint8_t* src = head + page * page_bytes + (mine & ((1 << upp_log) - 1)) * C::UNIT;
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         stages + put * C::STAGE + lane * C::UNIT),
                     "l"(src), "r"(whole ? units * C::UNIT : C::UNIT), "r"(b)
                     : "memory");
      }
      put = put + 1 == C::STAGES ? 0 : put + 1;
      ask_u += units;
      --to_ask;
      if (++ask.s == ask.n) {
        const int b = ask.b;
        next_job<C::JOB>(p, before, ask, to_ask);
        head = head_of();
        ask_u = 0;
        if (ask.b != b) {
          entry_0 = INT_MIN;
          if (to_ask > 0) ask_len = units_of(a, ask.b);
        }
      }
    };
    for (int i = 0; i < C::STAGES && to_ask > 0; ++i) request();

    while (rest > 0 && ok) {
      // one job's units, or this warp's share of them
      const int job = use.b * p.pl.jobs_per_seq + use.job;
      const long long slot = (long long)job + worker;
      const int hk = use.job / p.pl.blocks, row0 = use.job % p.pl.blocks * (8 * NT);
      const int len = a.len[use.b];
      const int end = use.n - use.s < rest ? use.n : use.s + (int)rest;
      if (lane == 0 && use.s == 0) p.span[job].x = worker;
      if (lane == 0 && end == use.n) p.span[job].y = worker;

      // q as an operand: row g of a block of 8, a group's channels 8 t .. 8 t + 7, as
      // fp16 with the row's largest value between 2^9 and 2^10 (what that rounds is at most
      // 2^-34 of it); channels that meet codes at place 3 16 times that.  base: what the 8s
      // add to this lane's two rows, taken off.
      uint4 q[QREG ? NT : 1][QREG ? R : 1];
      float2 base[BREG ? R : 1];
      uint8_t* const qs = ring + C::WARPS * C::STAGES * C::STAGE + warp * (C::QBYTES + C::BBYTES + C::SBYTES);
      float2* const bs = reinterpret_cast<float2*>(qs + C::QBYTES) + (WIDE ? g : t);
      uint32_t* const aside = reinterpret_cast<uint32_t*>(qs + C::QBYTES + C::BBYTES);
      float scale[2];                        // of this lane's rows' scores
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = row0 + 8 * n + g;
        const long long at = (long long)use.b * a.steps + row / p.pl.G;
        const uint16_t* from = a.q + (at * a.h_q + hk * p.pl.G + row % p.pl.G) * D + 8 * t;
        uint4 raw[R];
        uint32_t most2 = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          raw[r] = row < p.pl.R ? *reinterpret_cast<const uint4*>(from + 32 * r) : make_uint4(0, 0, 0, 0);
          most2 = max_u16x2(max_u16x2(most2, raw[r].x & 0x7fff7fffu), raw[r].y & 0x7fff7fffu);
          most2 = max_u16x2(max_u16x2(most2, raw[r].z & 0x7fff7fffu), raw[r].w & 0x7fff7fffu);
        }
        most2 = max(most2 & 0xffffu, most2 >> 16);     // (an infinity or a NaN: 0x7f80 or above)
        most2 = max(most2, __shfl_xor_sync(0xffffffffu, most2, 1));
        most2 = max(most2, __shfl_xor_sync(0xffffffffu, most2, 2));
        const float most = __uint_as_float(most2 << 16);
        // 2^9 over the power of two in `most`, at most 2^120 (a row of nothing but tiny numbers)
        const uint32_t ex = min(263 - min((int)(__float_as_uint(most) >> 23), 254), 247);
        const uint32_t up = ex << 7 | ex << 23, up16 = (ex + 4) << 7 | (ex + 4) << 23;   // bf16 pairs
        const float down = p.qscale * pow2(-kUnit7) * __uint_as_float((254 - ex) << 23);
        if constexpr (WIDE) {
          scale[n] = down;
        } else {
          scale[0] = __shfl_sync(0xffffffffu, down, 8 * t);
          scale[1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const uint4 h = make_uint4(half_pair(raw[r].x, up16), half_pair(raw[r].y, up), half_pair(raw[r].z, up16),
                                     half_pair(raw[r].w, up));
          if constexpr (QREG) q[n][r] = h;
          else *reinterpret_cast<uint4*>(qs + (n * R + r) * 512 + lane * 16) = h;
        }
      }
      const auto q_at = [&](int n, int r) {
        if constexpr (QREG) return q[n][r];
        else return *reinterpret_cast<const uint4*>(qs + (n * R + r) * 512 + lane * 16);
      };
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint4 x = q_at(0, r), y = q_at(NT - 1, r);   // (a lane reads what it wrote)
        float c[4];
        float2 sums;
        if constexpr (WIDE) {
          const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
          mma(c, a0, kLess8At3, kLess8At7, 0.0f, 0.0f, 0.0f, 0.0f);
          mma(c, a1, kLess8At3, kLess8At7);
          sums = make_float2(c[0], c[2]);
        } else {
          const uint32_t less8[4] = {kLess8At3, kLess8At3, kLess8At7, kLess8At7};
          mma(c, less8, x.x, x.y, 0.0f, 0.0f, 0.0f, 0.0f);
          mma(c, less8, x.z, x.w);
          sums = make_float2(c[0], c[1]);
        }
        if constexpr (BREG) base[r] = sums;
        else if ((WIDE ? t : g) == 0) bs[r * 8] = sums;
      }
      if constexpr (!BREG) __syncwarp();
      // the last token that this lane's rows see
      int last[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        last[i] = len - a.steps + min((row0 + (WIDE ? 8 * i + g : 2 * t + i)) / p.pl.G, a.steps - 1);
      const int all_see = len - a.steps;     // tokens up to this one are every row's
      Sums<D, NT> m;
      m.v = kLeastV;
      m.fresh = 3;
      m.stands = false;
      m.ref[0] = m.ref[1] = m.sum[0] = m.sum[1] = 0.0f;
      uint32_t poison = 0;                   // this lane's rows' groups that are NaN, eight bits a row
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int x = 0; x < 2 * NT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) m.o[r][x][e] = 0.0f;
      float* const part = p.part + slot * (8 * NT) * D;
      float2* const ml = p.ml + slot * (8 * NT);

      // Where not every row sees all of a stage's tokens: in tokens of no row (past the
      // sequence, of a page that is not there) V's scales become zeros,
      // whatever the cache holds.  So do scales that are not finite, for a row that does not see
      // the token gives it a weight of zero, and its product with them would be NaN; groups of
      // rows that do see it are noted and become NaN at the end.
      const auto clean = [&](int u, uint8_t* st, uint32_t gone) {
#pragma unroll 1
        for (int i = 0; i < 2 * C::UNITS; ++i) {
          const int token = u * kv4::kUnit + 8 * i + g;
          uint8_t* at = st + i / 2 * C::UNIT + 16 * D + (g + i % 2 * 8) * (D / 8) + D / 16 + t % (R / 2) * 4;
          uint32_t w = *reinterpret_cast<const uint32_t*>(at), odd = 0;
          if ((w & 0x7f80u) == 0x7f80u) odd |= 1u, w &= 0xffff0000u;
          if ((w & 0x7f800000u) == 0x7f800000u) odd |= 2u, w &= 0xffffu;
          if (token >= len || gone >> (i / 2) & 1) w = odd = 0;
          *reinterpret_cast<uint32_t*>(at) = w;
          for (uint32_t lanes = __ballot_sync(0xffffffffu, odd != 0); lanes != 0; lanes &= lanes - 1) {
            const int from = __ffs(lanes) - 1;
            const int which = __shfl_sync(0xffffffffu, token, from);
            const uint32_t groups = __shfl_sync(0xffffffffu, odd << (2 * (t % (R / 2))), from);
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (which <= last[k]) poison |= groups << (8 * k);
          }
        }
        __syncwarp();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the stage's next copy
      };

      // A stage of units from u on; none: the first, the sums are zero.
      const auto meet = [&](int u, uint8_t* st, uint32_t gone, bool edge, bool none) {
        constexpr int NU = C::UNITS;
        constexpr int SET = kSet<D>, TOKS = kTokens<NT>;
        float s[NU][NT][4];                  // scores: token_of(x, e) of each unit, row row_of<NT>(e)
#pragma unroll
        for (int k = 0; k < NU; ++k) {
          uint32_t ks[TOKS][R / 2];          // two groups a word
#pragma unroll
          for (int i = 0; i < TOKS; ++i) words_at<R / 2>(ks[i], scales_of<D, NT>(st, lane, k, i));
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[k][x][e] = 0.0f;
#pragma unroll
          for (int set = 0; set < R / SET; ++set) {
            uint32_t w0[SET], w1[SET];
            codes_at<D>(w0, w1, st + k * C::UNIT, lane, set);
#pragma unroll
            for (int rr = 0; rr < SET; ++rr) {
              const int r = set * SET + rr;
              const uint32_t x1 = __funnelshift_r(w0[rr], w0[rr], 8), y1 = __funnelshift_r(w1[rr], w1[rr], 8);
              float sc[TOKS];
#pragma unroll
              for (int i = 0; i < TOKS; ++i) sc[i] = r % 2 ? hi_f32(ks[i][r / 2]) : lo_f32(ks[i][r / 2]);
              const uint4 qx = q_at(0, r);
              float2 bb;
              if constexpr (BREG) bb = base[r];
              else bb = bs[r * 8];
              float c[NT][4];
              if constexpr (WIDE) {          // rows by tokens
                const uint4 qy = q_at(1, r);
                const uint32_t a0[4] = {qx.x, qy.x, qx.y, qy.y}, a1[4] = {qx.z, qy.z, qx.w, qy.w};
                mma(c[0], a0, w0[rr] & kAt3, w0[rr] & kAt7, bb.x, bb.x, bb.y, bb.y);
                mma(c[1], a0, w1[rr] & kAt3, w1[rr] & kAt7, bb.x, bb.x, bb.y, bb.y);
                mma(c[0], a1, x1 & kAt3, x1 & kAt7);
                mma(c[1], a1, y1 & kAt3, y1 & kAt7);
              } else {                       // tokens by rows
                const uint32_t f0[4] = {w0[rr] & kAt3, w1[rr] & kAt3, w0[rr] & kAt7, w1[rr] & kAt7};
                const uint32_t f1[4] = {x1 & kAt3, y1 & kAt3, x1 & kAt7, y1 & kAt7};
                mma(c[0], f0, qx.x, qx.y, bb.x, bb.y, bb.x, bb.y);
                mma(c[0], f1, qx.z, qx.w);
              }
#pragma unroll
              for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[k][x][e] = fmaf(c[x][e], sc[WIDE ? 2 * x + e % 2 : e / 2], s[k][x][e]);
            }
          }
        }
        // V's scales: twice their magnitudes' bits (a word's first sign falls into its second's last
        // place, which does not count here) less those of 2^(v - kNarrow), the smaller ones wrapped
        // around to above all
        uint32_t far = 0;
        const uint32_t from = ((0u - 2 * bf16_pow2(m.v - kNarrow)) & 0xffffu) * 0x10001u;
#pragma unroll
        for (int i = 0; i < C::WORDS / C::RUN; ++i) {
          uint32_t w[C::RUN];
          words_at<C::RUN>(w, reinterpret_cast<uint8_t*>(v_scales<D, NT>(st, lane, i)));
#pragma unroll
          for (int k = 0; k < C::RUN; ++k) far = __viaddmax_u16x2(w[k] + w[k], from, far);
        }
        far = max(far & 0xffffu, far >> 16);
        const bool odd = far >= 2 * 128 * (kWide + kNarrow);   // (or zero)
        bool over = m.fresh != 0;
        const float room = kTop + kGrow - (float)m.v;
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[k][x][e] = fmaf(s[k][x][e], scale[row_of<NT>(e)], -m.ref[row_of<NT>(e)]);
        if (edge) {
#pragma unroll
          for (int k = 0; k < NU; ++k) {
            const int at = gone >> k & 1 ? 0x7fffffff - 16 : (u + k) * kv4::kUnit;
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (at + token_of<NT>(lane, x, e) > last[row_of<NT>(e)]) s[k][x][e] = -INFINITY;
          }
        }
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) over = over || s[k][x][e] > room;
        if (__any_sync(0xffffffffu, over || odd)) {
          bool apart;
          int top = 0;
          const int v0 = m.v, v1 = range_of<D, NT>(st, lane, v0, apart, top);
          if (v1 != v0 || __any_sync(0xffffffffu, over)) move_refs(m, s, v1);
          if (apart || (v1 != v0 && !none)) {
            // V's scales are far apart, or far from those before: what there is goes to the slot, and
            // those that do not lie near the largest do too, those near each other at a time
            put_sums(m, v0, part, ml, lane);
            m.stands = true;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int x = 0; x < 2 * NT; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) m.o[r][x][e] = 0.0f;
            if (apart) {
              float y[NU][NT][4];
#pragma unroll
              for (int k = 0; k < NU; ++k)
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                  for (int e = 0; e < 4; ++e) y[k][x][e] = ex2(s[k][x][e]);
              // those near 2^v1 stay in the stage
              const uint32_t lo = bf16_pow2(v1 - kNarrow), hi = top <= v1 + kWide ? 0x7f80u : lo;
              uint32_t most = leave<D, NT>(st, aside, lane, lo, hi, 0, true);
              if (hi != lo) top = above(most);
              else most = lo;                // all that there is goes to the slot
              while (most != 0) {
                most = leave<D, NT>(st, aside, lane, bf16_pow2(top - kNarrow), bf16_pow2(top), v1 - top, false);
                add_to_slot<D, NT>(y, st, top, part, lane);
                top = above(most);
              }
              leave<D, NT>(st, aside, lane, lo, hi, 0, false);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[k][x][e] = ex2(s[k][x][e]);
        add_weights(m, s);
        add_values(m, s, st, lane);
      };

#pragma unroll 1
      for (int s = use.s; s < end; ++s) {
        const int u = s * C::UNITS;
        if (!__all_sync(0xffffffffu, try_wait(bar + get, parity)))
          ok = __all_sync(0xffffffffu, tc::mbar_wait(bar + get, parity, kWaitClocks));
        if (!ok) break;
        uint8_t* st = ring + (warp * C::STAGES + get) * C::STAGE;
        const uint32_t gone = bad >> (get * C::UNITS) & ((1u << C::UNITS) - 1);
        const bool edge = (u + C::UNITS) * kv4::kUnit - 1 > all_see || gone != 0;
        if (edge) clean(u, st, gone);
        meet(u, st, gone, edge, s == use.s);
        __syncwarp();
        get = get + 1 == C::STAGES ? 0 : get + 1;
        parity ^= get == 0;
        if (to_ask > 0) request();
      }
      if (__any_sync(0xffffffffu, poison != 0)) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int x = 0; x < 2 * NT; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (poison >> (8 * row_of<NT>(e) + r) & 1) m.o[r][x][e] = __uint_as_float(0x7fc00000u);
      }
      put_sums(m, m.v, part, ml, lane);      // the share's sums into its slot
      if (!ok) break;
      rest -= end - use.s;
      use.s = end;
      if (end == use.n) next_job<C::JOB>(p, before, use, rest);
    }
    if (!ok) {                               // a copy did not come: wait for the others, then leave
      if (lane == 0) record_status(a.status, GDN_ERR_DEVICE_TIMEOUT);
      for (int i = 1; i < C::STAGES; ++i) {
        get = get + 1 == C::STAGES ? 0 : get + 1;
        parity ^= get == 0;
        if (get == put) break;               // stages from here on hold nothing asked for
        tc::mbar_wait(bar + get, parity, kWaitClocks);
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

constexpr int kJoinThreads = 256, kMaxJoinThreads = 1024;

// Joins the shares of each row: 2^(ref_i - M) of each, over the sum of the sums.  A CTA
// takes threads / LANES / groups rows (of up to 128 channels), `groups` (a power of two) lane
// groups to a row, each every groups-th share with four shares' loads in flight.
template <int D, int NT>
__global__ void __launch_bounds__(kMaxJoinThreads) attn_kv4_join(Kv4Params p, int groups) {
  constexpr int LANES = D / 4 < 32 ? D / 4 : 32, CHUNKS = D / 4 / LANES;
  __shared__ float4 acc[kMaxJoinThreads];
  __shared__ float2 stat[kMaxJoinThreads];
  const AttnKv4Args& a = p.a;
  const int per = blockDim.x / LANES / groups;   // rows of a CTA
  const int set = threadIdx.x / LANES, grp = set % groups;
  const long long item = (long long)blockIdx.x * per + set / groups, items = (long long)a.batch * a.steps * a.h_q * CHUNKS;
  const bool mine = item < items;
  const int c4 = mine ? (int)(item % CHUNKS) * LANES + threadIdx.x % LANES : 0;
  const long long out_row = mine ? item / CHUNKS : 0;         // [b][step][h]
  const int h = (int)(out_row % a.h_q), tok = (int)(out_row / a.h_q);
  const int b = tok / a.steps, step = tok - b * a.steps;
  const int hk = h / p.pl.G, row = step * p.pl.G + h - hk * p.pl.G;
  const int job = b * p.pl.jobs_per_seq + hk * p.pl.blocks + row / (8 * NT);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  uint2 gt = make_uint2(0, 0);
  if (mine && a.gate && grp == 0)              // on its way under the sums
    gt = *reinterpret_cast<const uint2*>(a.gate + (long long)tok * a.gate_st + h * a.gate_sh + 4 * c4);
  const int len = a.len[b];
  const bool any = mine && units_of(a, b) > 0;
  float M = -INFINITY, L = 0.0f;
  float4 o = make_float4(0, 0, 0, 0);
  const auto add = [&](float m, float l, const float4& v) {
    if (l == 0.0f) return;                     // saw nothing (a NaN sum counts)
    const float to = fmaxf(M, m), f = ex2(M - to), e = ex2(m - to);
    L = L * f + l * e;
    o.x = o.x * f + v.x * e;
    o.y = o.y * f + v.y * e;
    o.z = o.z * f + v.z * e;
    o.w = o.w * f + v.w * e;
    M = to;
  };
  if (any) {
    const int2 span = p.span[job];
    const Ranges own = ranges_of(span.x, span.y, p.pl.workers);
    const long long at = ((long long)job + own.first) * (8 * NT) + row % (8 * NT);
    const float2* ml = p.ml + at;
    const float4* part = reinterpret_cast<const float4*>(p.part + at * D) + c4;
    for (int i = grp; i < own.count; i += 4 * groups) {
      float2 m[4];
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int x = i + k * groups;
        m[k] = make_float2(0.0f, 0.0f);
        if (x < own.count) {
          m[k] = ml[(long long)x * (8 * NT)];
          v[k] = part[(long long)x * (8 * NT) * (D / 4)];
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) add(m[k].x, m[k].y, v[k]);
    }
  }
  for (int half = groups / 2; half > 0; half /= 2) {   // halves of the groups hand over to the others
    if (grp >= half && grp < 2 * half) {
      acc[threadIdx.x] = o;
      stat[threadIdx.x] = make_float2(M, L);
    }
    __syncthreads();
    if (grp < half) add(stat[threadIdx.x + half * LANES].x, stat[threadIdx.x + half * LANES].y, acc[threadIdx.x + half * LANES]);
  }
  if (!mine || grp != 0) return;
  // no token seen: zeros; tokens seen whose weights are all zero (scores of -inf): NaN
  const bool sees = any && len - (a.steps - 1 - step) > 0;
  const float inv = !sees ? 0.0f : L == 0.0f ? __uint_as_float(0x7fc00000u) : 1.0f / L;
  float r[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
  if (a.gate) {
    r[0] *= sigmoid(lo_f32(gt.x));
    r[1] *= sigmoid(hi_f32(gt.x));
    r[2] *= sigmoid(lo_f32(gt.y));
    r[3] *= sigmoid(hi_f32(gt.y));
  }
  *reinterpret_cast<uint2*>(a.out + out_row * D + 4 * c4) = make_uint2(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]));
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// One block of 8 rows at a time, or two where there are more than 8.
int row_blocks(int rows) { return rows <= 8 ? 1 : 2; }

size_t slots(int batch, int jobs_per_seq) { return (size_t)batch * jobs_per_seq + (size_t)kMaxCtas * kMaxWarps; }

template <int D, int NT>
cudaError_t launch_n(const AttnKv4Args& a, cudaStream_t stream, int sms) {
  using C = Cfg<D, NT>;
  static_assert(C::WARPS <= kMaxWarps, "workspace");
  Kv4Params p;
  p.a = a;
  p.pl.G = a.h_q / a.h_kv;
  p.pl.R = a.steps * p.pl.G;
  p.pl.blocks = (p.pl.R + 8 * NT - 1) / (8 * NT);
  p.pl.jobs_per_seq = a.h_kv * p.pl.blocks;
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  p.pl.workers = ctas * C::WARPS;
  p.qscale = a.scale * 1.4426950408889634f;
  char* ws = static_cast<char*>(a.scratch);
  p.span = reinterpret_cast<int2*>(ws);
  ws += up256((size_t)a.batch * p.pl.jobs_per_seq * sizeof(int2));
  const size_t rows = slots(a.batch, p.pl.jobs_per_seq) * 8 * NT;
  p.ml = reinterpret_cast<float2*>(ws);
  ws += up256(rows * sizeof(float2));
  p.part = reinterpret_cast<float*>(ws);
  const auto kernel = attn_kv4_kernel<D, NT>;
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess) return e;
  cudaLaunchAttribute overlap;
  overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  overlap.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(C::WARPS * 32);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kernel, p)) != cudaSuccess) return e;
  // Lane groups to a row: one for every four shares that a job can have where all are alike; larger
  // CTAs where there are few rows with many shares (four sequences of up to 4000 10.6 us for 12.3;
  // with few shares they only start later, one of 833 9.3 for 8.7).
  constexpr int LANES = D / 4 < 32 ? D / 4 : 32;
  const long long items = (long long)a.batch * a.steps * a.h_q * (D / 4 / LANES);
  const long long stages = ((long long)a.width * a.page / kv4::kUnit + C::UNITS - 1) / C::UNITS;
  const long long even = p.pl.workers / ((long long)a.batch * p.pl.jobs_per_seq) + 1, shares = stages < even ? stages : even;
  const int threads = items < sms && shares > 4 * kJoinThreads / LANES ? kMaxJoinThreads : kJoinThreads;
  int groups = 1;
  while (groups < threads / LANES && 4 * groups < shares) groups *= 2;
  const long long per = threads / LANES / groups;
  cfg.gridDim = dim3((unsigned)((items + per - 1) / per));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attn_kv4_join<D, NT>, p, groups);
}

template <int D>
cudaError_t launch_d(const AttnKv4Args& a, cudaStream_t stream, int sms) {
  return row_blocks(a.steps * (a.h_q / a.h_kv)) == 1 ? launch_n<D, 1>(a, stream, sms) : launch_n<D, 2>(a, stream, sms);
}

}  // namespace

size_t attn_kv4_scratch_bytes(int batch, int steps, int h_q, int h_kv, int d) {
  const int rows = steps * (h_q / h_kv), per = 8 * row_blocks(rows);
  const size_t n = slots(batch, h_kv * ((rows + per - 1) / per)) * per;
  return up256((size_t)batch * (h_kv * ((rows + per - 1) / per)) * sizeof(int2)) + up256(n * sizeof(float2)) +
         up256(n * d * sizeof(float));
}

cudaError_t launch_attn_kv4(const AttnKv4Args& p, cudaStream_t stream) {
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
