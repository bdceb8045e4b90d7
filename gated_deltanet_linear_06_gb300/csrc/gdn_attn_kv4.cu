// gdn_attn_kv4.cu -- attention of a batch of sequences over the 4-bit paged cache.
#include <math.h>

#include "../../include/gdn.h"
#include "gdn_kv4.cuh"
#include "gdn_launch.h"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr long long kWaitClocks = 2000000000LL;   // a second or so: a copy that has not come by then never will
constexpr float kSlack = 20.0f;                    // binary orders between a row's reference and its maximum
constexpr int kMinItems = 2;                       // units that a warp takes at least
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
  long long* before;         // [batch + 1] units of the sequences before each
  float2* ml;                // per slot and row: (reference, sum)
  float* part;               // per slot and row: d sums
};

// Rows (of 8) that a warp takes at once: two blocks where there are that many rows and
// the accumulators leave room.
template <int D, int NT>
struct Cfg {
  static constexpr int WARPS = D == 256 ? 8 : (NT == 1 ? 16 : 12);
  static constexpr int STAGE = kv4::unit_bytes(D);
  static constexpr int STAGES = D == 256 ? 5 : (D == 128 ? (NT == 1 ? 5 : 7) : (NT == 1 ? 10 : 12));
  static constexpr int SMEM = WARPS * STAGES * STAGE;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Two codes, at bits 3..6 and 19..22 of x, as bf16 values code - 8: with the exponent of
// 16 the bits read 16 + code, and 24 is taken off exactly.
__device__ __forceinline__ uint32_t values(uint32_t x) {
  uint32_t y;
  asm("lop3.b32 %0, %1, 0x00780078, 0x41804180, 0xea;" : "=r"(y) : "r"(x));   // (x & mask) | base
  asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(y) : "r"(0x41c041c0u));
  return y;
}

__device__ __forceinline__ float lo_f32(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f32(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Length of sequence b, in units; a length out of range counts as none.
__device__ __forceinline__ int units_of(const AttnKv4Args& a, int b) {
  const int n = a.len[b];
  return n > 0 && n <= (long long)a.width * a.page ? (n + kv4::kUnit - 1) / kv4::kUnit : 0;
}

// before[0 .. batch] in shared memory, by the whole CTA.
__device__ void sum_units(const AttnKv4Args& a, long long* before, long long* warp_sums, bool report) {
  const int threads = blockDim.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int per = (a.batch + threads - 1) / threads, b0 = threadIdx.x * per;
  long long mine = 0;
  for (int i = 0; i < per; ++i)
    if (b0 + i < a.batch) {
      const int n = a.len[b0 + i];
      if (report && (n < 0 || n > (long long)a.width * a.page)) record_status(a.status, GDN_ERR_DEVICE_BOUNDS);
      mine += units_of(a, b0 + i);
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
      at += units_of(a, b0 + i);
      if (b0 + i == a.batch - 1) before[a.batch] = at;
    }
  __syncthreads();
}

// Warps that take part: one for every kMinItems items at most, so that none is empty.
__device__ __forceinline__ int workers_of(const Kv4Params& p, long long total) {
  const long long n = (total + kMinItems - 1) / kMinItems;
  return n < p.pl.workers ? (int)n : p.pl.workers;
}

// Where an item (a unit of a job) lies.
struct Item {
  int b, job, u, n;          // sequence, job of it, unit, units of the sequence
};

__device__ __forceinline__ void next_item(const Kv4Params& p, const long long* before, Item& it) {
  if (++it.u < it.n) return;
  it.u = 0;
  if (++it.job < p.pl.jobs_per_seq) return;
  it.job = 0;
  do {
    ++it.b;
    it.n = it.b < p.a.batch ? (int)(before[it.b + 1] - before[it.b]) : 0;
  } while (it.n == 0 && it.b < p.a.batch);
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::WARPS * 32, 1) attn_kv4_kernel(Kv4Params p) {
  using C = Cfg<D, NT>;
  constexpr int R = D / 32;                  // groups
  constexpr int NV = D / 64;                 // vectors of a lane
  constexpr bool QREG = NT * R <= 8;
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
  sum_units(a, before, warp_sums, blockIdx.x == 0);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= a.batch; b += blockDim.x) p.before[b] = before[b];

  // This warp's items, and where the first one is.
  const long long total = before[a.batch] * p.pl.jobs_per_seq;
  const int worker = warp * gridDim.x + blockIdx.x;   // few workers: on many SMs
  const int workers = workers_of(p, total);
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
      use.n = (int)(before[lo + 1] - before[lo]);
      const long long rest = x0 - before[lo] * p.pl.jobs_per_seq;
      use.job = (int)(rest / use.n);
      use.u = (int)(rest - (long long)use.job * use.n);
    }
    Item ask = use;
    long long asked = x0;
    const int upp = a.page / kv4::kUnit;     // units of a page
    int entry = 0, entry_b = -1, entry_0 = 0;   // this lane's of 32 entries of a sequence's table
    uint32_t bad = 0;                        // stages whose page there is not
    const uint32_t ring0 = tc::smem_u32(ring) + warp * C::STAGES * C::STAGE;
    int put = 0, get = 0;
    uint32_t parity = 0;

    const auto request = [&]() {             // one more unit into the ring
      const int pg = ask.u / upp;
      if (ask.b != entry_b || pg < entry_0 || pg >= entry_0 + 32) {
        entry_b = ask.b;
        entry_0 = pg;
        entry = pg + lane < a.width ? a.table[(long long)ask.b * a.width + pg + lane] : -1;
      }
      const int page = __shfl_sync(0xffffffffu, entry, pg - entry_0);
      const bool there = page >= 0 && page < a.n_pages;
      if (!there && lane == 0) record_status(a.status, GDN_ERR_DEVICE_BOUNDS);
      bad = there ? bad & ~(1u << put) : bad | 1u << put;
      if (there && lane == 0) {
        const uint8_t* src = a.cache + (((long long)page * a.h_kv + ask.job / p.pl.blocks) * upp + ask.u % upp) * C::STAGE;
        const uint32_t b = tc::smem_u32(bar + put);
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(b), "r"(C::STAGE) : "memory");
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                ring0 + put * C::STAGE),
            "l"(src), "r"(C::STAGE), "r"(b)
            : "memory");
      } else if (lane == 0) {                // nothing comes: the stage's turn ends at once
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(bar + put)) : "memory");
      }
      put = put + 1 == C::STAGES ? 0 : put + 1;
      ++asked;
      next_item(p, before, ask);
    };
    while (asked < x1 && asked < x0 + C::STAGES) request();

    long long x = x0;
    while (x < x1 && ok) {
      // one job's units, or this warp's share of them
      const long long slot = (long long)use.b * p.pl.jobs_per_seq + use.job + worker;
      const int hk = use.job / p.pl.blocks, row0 = use.job % p.pl.blocks * (8 * NT);
      const int len = a.len[use.b];
      const long long left = x1 - x;
      const int end = use.n - use.u < left ? use.n : use.u + (int)left;
      // q as the second operand: row g of a block of 8, a group's channels 8 t .. 8 t + 7
      uint4 q[QREG ? NT : 1][QREG ? R : 1];
      const auto q_row = [&](int n, int r) -> uint4 {
        const int row = row0 + 8 * n + g;
        if (row >= p.pl.R) return make_uint4(0, 0, 0, 0);
        const long long at = (long long)use.b * a.steps + row / p.pl.G;
        return *reinterpret_cast<const uint4*>(a.q + (at * a.h_q + hk * p.pl.G + row % p.pl.G) * D + 32 * r + 8 * t);
      };
      if constexpr (QREG) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < R; ++r) q[n][r] = q_row(n, r);
      }
      // the last token that rows 2 t and 2 t + 1 of each block see
      int last[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) last[n][i] = len - a.steps + min((row0 + 8 * n + 2 * t + i) / p.pl.G, a.steps - 1);
      const int all_see = len - a.steps;     // tokens up to this one are seen by every row
      float o[NT][R][2][4], ref[NT][2], sum[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][r][i][e] = 0.0f;
        ref[n][0] = ref[n][1] = -3.402823466e38f;
        sum[n][0] = sum[n][1] = 0.0f;
      }

#pragma unroll 1
      for (int u = use.u; u < end; ++u, ++x) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(bar + get, parity, kWaitClocks));
        if (!ok) break;
        const uint8_t* st = ring + (warp * C::STAGES + get) * C::STAGE;
        if (!(bad >> get & 1)) {
          // scores: tokens g and g + 8 by rows 2 t, 2 t + 1
          float s[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
          const uint8_t* sc = st + 16 * D + g * (D / 8);
          uint32_t ks[2][R / 2], vs[2][R / 2];   // scales of tokens g and g + 8, two groups a word
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < R / 2; ++i) {
              ks[h][i] = *reinterpret_cast<const uint32_t*>(sc + h * D + 4 * i);
              vs[h][i] = *reinterpret_cast<const uint32_t*>(sc + h * D + R * 2 + 4 * i);
            }
          const uint4* kv = reinterpret_cast<const uint4*>(st) + lane;
#pragma unroll
          for (int v = 0; v < (NV + 1) / 2; ++v) {
            // words of token g and of token g + 8
            uint32_t w0[4], w1[4];
            if constexpr (NV == 1) {
              const uint4 x4 = kv[0];
              w0[0] = x4.x, w0[1] = x4.y, w1[0] = x4.z, w1[1] = x4.w;
            } else {
              const uint4 x4 = kv[v * 32], y4 = kv[(v + NV / 2) * 32];
              w0[0] = x4.x, w0[1] = x4.y, w0[2] = x4.z, w0[3] = x4.w;
              w1[0] = y4.x, w1[1] = y4.y, w1[2] = y4.z, w1[3] = y4.w;
            }
#pragma unroll
            for (int k = 0; k < (NV == 1 ? 2 : 4); ++k) {
              const int r = 4 * v + k;
              float c[NT][4];
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) c[n][e] = 0.0f;
              uint32_t f[2][4];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                f[i][0] = values(__funnelshift_r(w0[k], w0[k], 8 * i));
                f[i][1] = values(__funnelshift_r(w1[k], w1[k], 8 * i));
                f[i][2] = values(__funnelshift_r(w0[k], w0[k], 8 * i + 4));
                f[i][3] = values(__funnelshift_r(w1[k], w1[k], 8 * i + 4));
              }
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const uint4 qq = QREG ? q[QREG ? n : 0][QREG ? r : 0] : q_row(n, r);
                mma(c[n], f[0], qq.x, qq.y);
                mma(c[n], f[1], qq.z, qq.w);
              }
              const float s0 = r % 2 ? hi_f32(ks[0][r / 2]) : lo_f32(ks[0][r / 2]);
              const float s1 = r % 2 ? hi_f32(ks[1][r / 2]) : lo_f32(ks[1][r / 2]);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                s[n][0] = fmaf(c[n][0], s0, s[n][0]);
                s[n][1] = fmaf(c[n][1], s0, s[n][1]);
                s[n][2] = fmaf(c[n][2], s1, s[n][2]);
                s[n][3] = fmaf(c[n][3], s1, s[n][3]);
              }
            }
          }
          // weights
          const int j = u * kv4::kUnit + g;
          const bool edge = u * kv4::kUnit + kv4::kUnit - 1 > all_see;
          bool over = false;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[n][e] *= p.qscale;
              if (edge && j + e / 2 * 8 > last[n][e % 2]) s[n][e] = -INFINITY;
              over = over || s[n][e] > ref[n][e % 2];
            }
          if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float m = fmaxf(s[n][i], s[n][2 + i]);
#pragma unroll
                for (int k = 4; k <= 16; k <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
                if (m > ref[n][i]) {
                  const float to = m + kSlack, f = ex2(ref[n][i] - to);
                  ref[n][i] = to;
                  sum[n][i] *= f;
#pragma unroll
                  for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                      o[n][r][k][i] *= f;
                      o[n][r][k][2 + i] *= f;
                    }
                }
              }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[n][e] = ex2(s[n][e] - ref[n][e % 2]);
              sum[n][e % 2] += s[n][e];
            }
          // outputs: channels by rows, over the 16 tokens
          const uint4* vv = reinterpret_cast<const uint4*>(st + 8 * D) + lane;
#pragma unroll
          for (int v = 0; v < (NV + 1) / 2; ++v) {
            uint32_t w0[4], w1[4];
            if constexpr (NV == 1) {
              const uint4 x4 = vv[0];
              w0[0] = x4.x, w0[1] = x4.y, w1[0] = x4.z, w1[1] = x4.w;
            } else {
              const uint4 x4 = vv[v * 32], y4 = vv[(v + NV / 2) * 32];
              w0[0] = x4.x, w0[1] = x4.y, w0[2] = x4.z, w0[3] = x4.w;
              w1[0] = y4.x, w1[1] = y4.y, w1[2] = y4.z, w1[3] = y4.w;
            }
#pragma unroll
            for (int k = 0; k < (NV == 1 ? 2 : 4); ++k) {
              const int r = 4 * v + k;
              const float s0 = r % 2 ? hi_f32(vs[0][r / 2]) : lo_f32(vs[0][r / 2]);
              const float s1 = r % 2 ? hi_f32(vs[1][r / 2]) : lo_f32(vs[1][r / 2]);
              uint32_t f[2][4];
              f[0][0] = values(w0[k] << 3);
              f[0][1] = values(w0[k] >> 1);
              f[0][2] = values(w1[k] << 3);
              f[0][3] = values(w1[k] >> 1);
              f[1][0] = values(w0[k] >> 5);
              f[1][1] = values(w0[k] >> 9);
              f[1][2] = values(w1[k] >> 5);
              f[1][3] = values(w1[k] >> 9);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float e0 = s[n][0] * s0, e1 = s[n][1] * s0, e2 = s[n][2] * s1, e3 = s[n][3] * s1;
                if (edge) {                  // whatever the scale of a token that is not seen
                  if (j > last[n][0]) e0 = 0.0f;
                  if (j > last[n][1]) e1 = 0.0f;
                  if (j + 8 > last[n][0]) e2 = 0.0f;
                  if (j + 8 > last[n][1]) e3 = 0.0f;
                }
                const uint32_t b0 = transpose8(pack_bf16x2(e0, e1)), b1 = transpose8(pack_bf16x2(e2, e3));
                mma(o[n][r][0], f[0], b0, b1);
                mma(o[n][r][1], f[1], b0, b1);
              }
            }
          }
        }
        __syncwarp();
        get = get + 1 == C::STAGES ? 0 : get + 1;
        parity ^= get == 0;
        if (asked < x1) request();
      }
      // the share's sums into its slot
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float l = sum[n][i];
#pragma unroll
          for (int k = 4; k <= 16; k <<= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
          const long long row = slot * (8 * NT) + 8 * n + 2 * t + i;
          if (g == 0) p.ml[row] = make_float2(ref[n][i], l);
#pragma unroll
          for (int r = 0; r < R; ++r)
            *reinterpret_cast<float4*>(p.part + row * D + 32 * r + 4 * g) =
                make_float4(o[n][r][0][i], o[n][r][0][2 + i], o[n][r][1][i], o[n][r][1][2 + i]);
        }
      use.u = end - 1;
      next_item(p, before, use);
    }
    if (!ok) {                               // a copy did not come: wait for the others, then leave
      if (lane == 0) record_status(a.status, GDN_ERR_DEVICE_TIMEOUT);
      for (long long y = x + 1; y < asked; ++y) {
        get = get + 1 == C::STAGES ? 0 : get + 1;
        parity ^= get == 0;
        tc::mbar_wait(bar + get, parity, kWaitClocks);
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

constexpr int kJoinThreads = 256;

// Joins the shares of each row: 2^(ref_i - M) of each, over the sum of the sums.
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) attn_kv4_join(Kv4Params p) {
  constexpr int LANES = D / 4;
  constexpr int GROUPS = kJoinThreads / LANES;
  __shared__ float4 acc[kJoinThreads];
  __shared__ float2 stat[kJoinThreads];
  const AttnKv4Args& a = p.a;
  const int b = blockIdx.x / a.steps, step = blockIdx.x % a.steps, h = blockIdx.y;
  const int hk = h / p.pl.G, row = step * p.pl.G + h % p.pl.G;
  const int c4 = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long n_before = p.before[b], n = p.before[b + 1] - n_before;
  const long long total = p.before[a.batch] * p.pl.jobs_per_seq;
  const int job = hk * p.pl.blocks + row / (8 * NT);
  float M = -INFINITY, L = 0.0f;
  float4 o = make_float4(0, 0, 0, 0);
  const int seen = a.len[b] - (a.steps - 1 - step);
  if (n > 0) {
    const long long first_item = n_before * p.pl.jobs_per_seq + job * n;
    // the worker of item x: the last whose share begins at or before it
    const int workers = workers_of(p, total);
    const int w0 = (int)(((first_item + 1) * workers - 1) / total);
    const int w1 = (int)(((first_item + n) * workers - 1) / total);
    const long long slot0 = (long long)b * p.pl.jobs_per_seq + job;
    for (int w = w0 + grp; w <= w1; w += GROUPS) {
      const long long at = (slot0 + w) * (8 * NT) + row % (8 * NT);
      const float2 ml = p.ml[at];
      const float4 v = *reinterpret_cast<const float4*>(p.part + at * D + 4 * c4);
      if (ml.y == 0.0f) continue;            // saw nothing
      const float m = fmaxf(M, ml.x), f = ex2(M - m), e = ex2(ml.x - m);
      L = L * f + ml.y * e;
      o.x = o.x * f + v.x * e;
      o.y = o.y * f + v.y * e;
      o.z = o.z * f + v.z * e;
      o.w = o.w * f + v.w * e;
      M = m;
    }
  }
  acc[threadIdx.x] = o;
  stat[threadIdx.x] = make_float2(M, L);
  __syncthreads();
  if (grp != 0) return;
  for (int k = 1; k < GROUPS; ++k) {
    const float2 st = stat[k * LANES + c4];
    const float4 v = acc[k * LANES + c4];
    if (st.y == 0.0f) continue;
    const float m = fmaxf(M, st.x), f = ex2(M - m), e = ex2(st.x - m);
    L = L * f + st.y * e;
    o.x = o.x * f + v.x * e;
    o.y = o.y * f + v.y * e;
    o.z = o.z * f + v.z * e;
    o.w = o.w * f + v.w * e;
    M = m;
  }
  // no token seen: zeros; tokens seen whose weights are all zero (scores of -inf): NaN
  const float inv = seen <= 0 || n == 0 ? 0.0f : 1.0f / L;
  float r[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
  if (seen > 0 && n > 0 && L == 0.0f) r[0] = r[1] = r[2] = r[3] = __uint_as_float(0x7fc00000u);
  const long long tok = blockIdx.x;
  if (a.gate) {
    const uint2 gt = *reinterpret_cast<const uint2*>(a.gate + tok * a.gate_st + h * a.gate_sh + 4 * c4);
    r[0] *= sigmoid(lo_f32(gt.x));
    r[1] *= sigmoid(hi_f32(gt.x));
    r[2] *= sigmoid(lo_f32(gt.y));
    r[3] *= sigmoid(hi_f32(gt.y));
  }
  *reinterpret_cast<uint2*>(a.out + (tok * a.h_q + h) * D + 4 * c4) =
      make_uint2(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]));
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
  p.before = reinterpret_cast<long long*>(ws);
  ws += up256((size_t)(a.batch + 1) * sizeof(long long));
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
  cfg.gridDim = dim3(a.batch * a.steps, a.h_q);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attn_kv4_join<D, NT>, p);
}

template <int D>
cudaError_t launch_d(const AttnKv4Args& a, cudaStream_t stream, int sms) {
  return row_blocks(a.steps * (a.h_q / a.h_kv)) == 1 ? launch_n<D, 1>(a, stream, sms) : launch_n<D, 2>(a, stream, sms);
}

}  // namespace

size_t attn_kv4_scratch_bytes(int batch, int steps, int h_q, int h_kv, int d) {
  const int rows = steps * (h_q / h_kv), per = 8 * row_blocks(rows);
  const size_t n = slots(batch, h_kv * ((rows + per - 1) / per)) * per;
  return up256((size_t)(batch + 1) * sizeof(long long)) + up256(n * sizeof(float2)) + up256(n * d * sizeof(float));
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
