// gdn_moe.cu -- a whole mixture-of-experts layer for a few tokens, in two
// kernels (HBM-bound: every chosen expert's weights are read once).
//
// Mathematics.  With few tokens each weight meets one or a few of them, so the
// layer costs its weights' bytes: 6 hidden inter per expert that any token
// chose.  The products run on the tensor cores all the same (m16n8k16: 16
// weight rows by 8 tokens), because their cost then does not grow with the
// tokens that share an expert.
//
// Kernel 1, router logits: a warp per (expert, 8 tokens).  The chosen experts
// hang on which logits are larger, so the sums are compensated: each lane adds
// its products to S, which starts at a constant so large that it rounds them to
// a coarse grid exactly, and what S drops goes to a second sum.  Logits stay
// pairs of fp32 from there on (fp64 additions run at 1/64 of the rate here: with
// them the choice of 8 experts alone took 12 us).
//
// Kernel 2, one CTA of 12 warps per SM, everything else:
//   - the choice of experts, by every CTA for itself, which is cheaper than a
//     grid barrier;
//   - phase 1, tiles of 8 gate rows over the same 8 up rows, so that silu(g) u
//     forms in one thread; columns are the expert's own tokens; four warps share
//     a tile, each with every fourth chunk of 128 weight columns;
//   - a grid barrier;
//   - phase 2, up to 16 output rows per CTA for ALL experts, so that a token's
//     experts add up in registers without atomics or partial results; columns
//     are tokens by their number, a group of 8 that an expert does not serve is
//     skipped; the CTA's warps deal out the chunks of 128 weight columns.
// Every warp feeds itself: it has three stages of 4 KB (16 rows x 128 columns, by
// TMA, 128-byte swizzle) and refills a stage as soon as it has multiplied it, so
// 12 warps keep some 100 KB on their way and no warp waits for another's data.
// The stages run ahead past the choice (the shared expert's weights load while
// kernel 1 runs) and past the grid barrier (the first down weights land during
// it).  (With one loading warp and stages that eight or sixteen warps multiplied
// together, every stage cost the latency of its activations and the meetings of
// the warps: 1500 clocks, where its bytes take 700.)
// Which warp adds what depends on the expert's and the chunk's numbers alone, so
// nothing in a token's arithmetic depends on the other tokens.
//
// The activations between the products are kept as two bf16 (16 bits of
// significand): one bf16 would cost 2^-9 of each, more than the fp32 output
// holds; the second product on the low half costs tensor time, not bytes.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_launch.h"
#include "gdn_prefill.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kTeam = 4, kTeams = 3, kMoeWarps = kTeam * kTeams, kMoeThreads = 32 * kMoeWarps;
constexpr int kCols = 128;                            // weight columns of a stage
constexpr uint32_t kStage = 16 * kCols * 2;
constexpr int kStages = 3;                            // of each warp
constexpr int kMaxExperts = 1024, kMaxPairs = GDN_MOE_MAX_TOKENS * 32;
constexpr long long kBarrierBudget = 1LL << 31;       // clock cycles

struct MoeSmem {
  uint64_t full[kMoeWarps][kStages];
  int n_active;
  int gave_up;                         // a wait ran out: no later one waits
  int scan_a[kMoeWarps], scan_p[kMoeWarps];
  float4 red[2][kMoeWarps][32];
  uint32_t mask[kMaxExperts][2];       // tokens of an expert
  uint16_t expert[kMaxExperts];        // active experts, ascending
  uint16_t base[kMaxExperts + 1];      // first pair of an active expert
  uint8_t turn[kMaxExperts];           // the warp that takes an active expert's first down chunk
  uint16_t rank[kMaxExperts];          // expert -> its place among the active
  float shared_w[GDN_MOE_MAX_TOKENS];  // the shared expert's factor
  uint16_t sel[kMaxPairs];             // chosen experts, token-major
  float sel_w[kMaxPairs];
  float pair_w[kMaxPairs];             // weights in the order of the pairs
  uint8_t pair_t[kMaxPairs];           // and their tokens
};
constexpr uint32_t kRing = kMoeWarps * kStages * kStage;
constexpr uint32_t kMoeSmem = kRing + sizeof(MoeSmem) + 1024;
static_assert(kMoeSmem <= 227 * 1024, "shared memory");

struct MoeMaps {
  CUtensorMap gate_up, gate_up_edge, down, down_edge, s_gate_up, s_gate_up_edge, s_down, s_down_edge;
};

struct MoeParams {
  MoeArgs a;
  float2* logit;        // [tokens][experts + 1], high and low part
  unsigned* barrier;    // arrivals of the grid barrier; zeroed by kernel 1
  uint16_t* act;        // [hi, lo][pairs][inter]
  uint16_t* s_act;      // [hi, lo][tokens][shared_inter]
  int rows3, tiles3;    // output rows per tile, tiles
};

// a + b as a rounded sum and its error (Knuth's two-sum).
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float s = a + b, bb = s - a;
  return make_float2(s, (a - (s - bb)) + (b - bb));
}

// ---- kernel 1 ----
// NT tokens per warp, UK steps of 256 columns with all their loads in flight.
template <int NT, int UK>
__global__ void __launch_bounds__(256) moe_router_kernel(const MoeParams p) {
  const MoeArgs& a = p.a;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.barrier = 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, unit = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int rows = a.experts + (a.s_gate ? 1 : 0), blocks = (a.tokens + NT - 1) / NT;
  if (unit >= rows * blocks) return;
  const int e = unit / blocks, t0 = (unit - e * blocks) * NT, nt = min(NT, a.tokens - t0);
  const uint16_t* w = (e < a.experts ? a.w_router + (size_t)e * a.hidden : a.s_gate) + lane * 8;
  const uint16_t* x[NT];
  constexpr float kGrid = 3072.0f;   // products go to S on a grid of 2^-12
  float S[NT], lo[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    x[t] = a.x + (size_t)(t0 + min(t, nt - 1)) * a.hidden + lane * 8;   // (the last token again past the end)
    S[t] = kGrid;
    lo[t] = 0.0f;
  }
  for (int k = 0; k < a.hidden; k += 256 * UK) {
    uint4 wv[UK], xv[UK][NT];
#pragma unroll
    for (int u = 0; u < UK; ++u) {
      const bool in = k + 256 * u + lane * 8 < a.hidden;
      wv[u] = in ? __ldg(reinterpret_cast<const uint4*>(w + k + 256 * u)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        xv[u][t] = in ? __ldg(reinterpret_cast<const uint4*>(x[t] + k + 256 * u)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < UK; ++u) {
      const uint32_t ww[4] = {wv[u].x, wv[u].y, wv[u].z, wv[u].w};
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t xx[4] = {xv[u][t].x, xv[u][t].y, xv[u][t].z, xv[u][t].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float wf = __uint_as_float(i & 1 ? ww[i >> 1] & 0xffff0000u : ww[i >> 1] << 16);
          const float xf = __uint_as_float(i & 1 ? xx[i >> 1] & 0xffff0000u : xx[i >> 1] << 16);
          const float s = fmaf(xf, wf, S[t]);
          lo[t] += fmaf(xf, wf, -(s - S[t]));   // exact: what S did not take
          S[t] = s;
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    // the lanes' pairs (S - grid, lo) join as pairs: the high parts' rounding is kept
    float h = S[t] - kGrid, l = lo[t];
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
      const float oh = __shfl_xor_sync(0xffffffffu, h, m), ol = __shfl_xor_sync(0xffffffffu, l, m);
      const float2 r = two_sum(h, oh);
      h = r.x;
      l = (l + ol) + r.y;
    }
    if (lane == 0 && t < nt) p.logit[(size_t)(t0 + t) * (a.experts + 1) + e] = two_sum(h, l);
  }
}

// ---- kernel 2 ----

// e^(v - top) for v <= top, both pairs: what the difference's rounding to fp32
// drops is put back as a factor (at -80 it alone would cost 2^-18 of the result).
__device__ __forceinline__ float exp_of(float2 v, float2 top) {
  const float2 d = two_sum(v.x, -top.x);
  return d.x < -200.0f ? 0.0f : expf(d.x) * (1.0f + (d.y + (v.y - top.y)));
}

// A 64-bit key in the order of the pairs, NaN lowest, -0 like 0.
__device__ __forceinline__ uint32_t order32(float v) {
  const uint32_t b = __float_as_uint(v == 0.0f ? 0.0f : v);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order32_value(uint32_t k) {
  return __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ unsigned long long order_key(float2 v) {
  return v.x != v.x ? 0ull : ((unsigned long long)order32(v.x) << 32) | order32(v.y == v.y ? v.y : 0.0f);
}
__device__ __forceinline__ float2 order_value(unsigned long long k) {
  return make_float2(order32_value((uint32_t)(k >> 32)), order32_value((uint32_t)k));
}

__device__ __forceinline__ void team_sync(int team) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * kTeam) : "memory");
}

__device__ __forceinline__ void tma3(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint64_t* mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(mbar))
      : "memory");
}
__device__ __forceinline__ void tma2(uint32_t dst, const CUtensorMap* tm, int x, int y, uint64_t* mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(tc::smem_u32(mbar))
      : "memory");
}

// After a wait that gave up, the CTA runs to its end without waiting (every warp
// still meets the others at their barriers); the status word tells.
__device__ __forceinline__ bool moe_wait(const MoeArgs& a, MoeSmem* sm, uint64_t* mbar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred P1;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 P1, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, P1;\n\t}\n"
      : "=r"(done)
      : "r"(tc::smem_u32(mbar)), "r"(parity)
      : "memory");
  if (done) return true;
  if (*reinterpret_cast<volatile int*>(&sm->gave_up)) return false;
  if (tc::mbar_wait(mbar, parity, kWaitBudget)) return true;
  *reinterpret_cast<volatile int*>(&sm->gave_up) = 1;
  record_status(a.status, GDN_ERR_DEVICE_TIMEOUT);
  return false;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 rows x 64 columns of weights by 8 tokens.  Each lane holds 8 columns in a
// row of A and of B, 16 bytes each, so that the columns of the four products
// are those of four lanes: a permutation of the columns, the same in both.
struct Frag {
  uint4 lo[2], hi[2];   // row g and row g + 8, column halves
};
__device__ __forceinline__ void mma_block(float (&c)[4], const Frag& f, const uint4 (&b)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    mma16816(c, f.lo[h].x, f.hi[h].x, f.lo[h].y, f.hi[h].y, b[h].x, b[h].y);
    mma16816(c, f.lo[h].z, f.hi[h].z, f.lo[h].w, f.hi[h].w, b[h].z, b[h].w);
  }
}

// 64 columns of one token's row from column k on, zeros past n: this lane's 16.
__device__ __forceinline__ void load_b(uint4 (&b)[2], const uint16_t* row, int k, int n, bool use) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    b[h] = use && k + 32 * h < n ? *reinterpret_cast<const uint4*>(row + k + 32 * h) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void load_b_cg(uint4 (&b)[2], const uint16_t* row, int k, int n, bool use) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    b[h] = use && k + 32 * h < n ? __ldcg(reinterpret_cast<const uint4*>(row + k + 32 * h)) : make_uint4(0, 0, 0, 0);
}

// Top-k of one token by one warp, into sel / sel_w; 32 V experts at most.
template <int V>
__device__ void choose(const MoeParams& p, MoeSmem* sm, int t, int lane) {
  const MoeArgs& a = p.a;
  const float2* lg = p.logit + (size_t)t * (a.experts + 1);
  unsigned long long key[V];
  unsigned long long best = 0;
  int at = -1;
#pragma unroll
  for (int j = 0; j < V; ++j) {   // every load in flight at once
    const int e = j * 32 + lane;
    key[j] = order_key(e < a.experts ? __ldcg(lg + e) : make_float2(0.0f, 0.0f));
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (j * 32 + lane < a.experts && (at < 0 || key[j] > best)) {
      best = key[j];
      at = j;
    }
  uint32_t used = 0;
  float2 top = make_float2(0.0f, 0.0f);
  float den = 0.0f, sum = 0.0f, mine = 0.0f;
  for (int k = 0; k < a.top_k; ++k) {
    const uint32_t hi = at >= 0 ? (uint32_t)(best >> 32) : 0, mh = __reduce_max_sync(0xffffffffu, hi);
    const bool c1 = at >= 0 && hi == mh;
    const uint32_t lo = c1 ? (uint32_t)best : 0, ml = __reduce_max_sync(0xffffffffu, lo);
    const bool c2 = c1 && lo == ml;
    const int e = (int)__reduce_min_sync(0xffffffffu, c2 ? (uint32_t)(at * 32 + lane) : 0xffffffffu);
    const float2 v = order_value(((unsigned long long)mh << 32) | ml);
    if (k == 0) {   // the softmax's maximum and sum
      top = v;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j * 32 + lane < a.experts) den += exp_of(order_value(key[j]), top);
      den = warp_sum(den);
    }
    const float w = exp_of(v, top);
    sum += w;
    if (lane == k) mine = w;
    if (lane == 0) {
      sm->sel[t * a.top_k + k] = (uint16_t)e;
      atomicOr(&sm->mask[e][t >> 5], 1u << (t & 31));
    }
    if ((e & 31) == lane) {
      used |= 1u << (e >> 5);
      best = 0;
      at = -1;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j * 32 + lane < a.experts && !(used >> j & 1) && (at < 0 || key[j] > best)) {
          best = key[j];
          at = j;
        }
    }
  }
  __syncwarp();
  if (lane < a.top_k) {
    const float w = mine / (a.renorm ? sum : den);
    sm->sel_w[t * a.top_k + lane] = w;
    if (t % (int)gridDim.x == (int)blockIdx.x) {
      if (a.topk_id) a.topk_id[t * a.top_k + lane] = sm->sel[t * a.top_k + lane];
      if (a.topk_w) a.topk_w[t * a.top_k + lane] = w;
    }
  }
  if (lane == 0 && a.s_gate) sm->shared_w[t] = sigmoid(__ldcg(lg + a.experts).x);
}

// Tokens of a mask below token t.
__device__ __forceinline__ int below(uint32_t m0, uint32_t m1, int t) {
  return t < 32 ? __popc(m0 & ((1u << t) - 1u)) : __popc(m0) + __popc(m1 & ((1u << (t - 32)) - 1u));
}

// The active experts in ascending order, their first pairs, and the pairs' weights.
__device__ void build_lists(const MoeParams& p, MoeSmem* sm, int tid) {
  const MoeArgs& a = p.a;
  const int warp = tid >> 5, lane = tid & 31;
  constexpr int PER = (kMaxExperts + kMoeThreads - 1) / kMoeThreads;
  int na = 0, np = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    if (e < a.experts) {
      const int n = __popc(sm->mask[e][0]) + __popc(sm->mask[e][1]);
      na += n > 0;
      np += n;
    }
  }
  int ia = na, ip = np;
  for (int m = 1; m < 32; m <<= 1) {
    const int oa = __shfl_up_sync(0xffffffffu, ia, m), op = __shfl_up_sync(0xffffffffu, ip, m);
    if (lane >= m) {
      ia += oa;
      ip += op;
    }
  }
  if (lane == 31) {
    sm->scan_a[warp] = ia;
    sm->scan_p[warp] = ip;
  }
  __syncthreads();
  ia -= na;
  ip -= np;
  int total = 0;
  for (int w = 0; w < kMoeWarps; ++w) {
    if (w < warp) {
      ia += sm->scan_a[w];
      ip += sm->scan_p[w];
    }
    total += sm->scan_a[w];
  }
  if (tid == 0) {
    sm->n_active = total;
    sm->base[total] = (uint16_t)(a.tokens * a.top_k);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    if (e < a.experts) {
      const int n = __popc(sm->mask[e][0]) + __popc(sm->mask[e][1]);
      if (n > 0) {
        sm->expert[ia] = (uint16_t)e;
        sm->base[ia] = (uint16_t)ip;
        sm->rank[e] = (uint16_t)ia;
        sm->turn[ia] = (uint8_t)((unsigned)e * (unsigned)((a.inter + kCols - 1) / kCols) % kMoeWarps);
        ++ia;
        ip += n;
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < a.tokens * a.top_k; i += kMoeThreads) {
    const int t = i / a.top_k, e = sm->sel[i];
    const int at = sm->base[sm->rank[e]] + below(sm->mask[e][0], sm->mask[e][1], t);
    sm->pair_w[at] = sm->sel_w[i];
    sm->pair_t[at] = (uint8_t)t;
  }
  __syncthreads();
}

template <int NG>   // groups of 8 tokens
__global__ void __launch_bounds__(kMoeThreads, 1)
    moe_experts_kernel(const __grid_constant__ MoeMaps maps, const __grid_constant__ MoeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const MoeArgs& a = p.a;
  const uint32_t raw = tc::smem_u32(smem), pad = (1024u - (raw & 1023u)) & 1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x, grid = gridDim.x;
  const int team = warp / kTeam, member = warp % kTeam;
  MoeSmem* sm = reinterpret_cast<MoeSmem*>(smem + pad + kRing);
  uint8_t* const ring = smem + pad + warp * kStages * kStage;          // this warp's
  const uint32_t ring_a = raw + pad + warp * kStages * kStage;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) tc::mbar_init(&sm->full[warp][s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 0) sm->gave_up = 0;
  for (int e = tid; e < a.experts; e += kMoeThreads) sm->mask[e][0] = sm->mask[e][1] = 0;
  __syncthreads();

  const int s_tiles = a.shared_inter >> 3, e_tiles = a.inter >> 3;   // 8-row tiles of an expert
  const int h_chunks = (a.hidden + kCols - 1) / kCols, tile_step = grid * kTeams;
  const int j0 = a.shared_inter > 0 ? -1 : 0;                        // expert -1 is the shared one
  int na = 0, n1 = s_tiles;                                          // active experts, phase 1 tiles
  const auto cols_of = [&](int j) { return j < 0 ? a.shared_inter : a.inter; };

  // This warp's stages in order: its chunks of its team's tiles, then its chunks
  // of the CTA's output tiles.  One walk loads, kStages ahead; one multiplies.
  struct Walk {
    int i, j, c;     // tile; expert (of phase 1: at the tile's change); chunk
  };
  const auto first1 = [&]() { return Walk{cta * kTeams + team, 0, member}; };
  const auto next1 = [&](Walk& w) {
    w.c += kTeam;
    if (w.c >= h_chunks) {
      w.c = member;
      w.i += tile_step;
    }
  };
  const bool any1 = member < h_chunks;   // this member has chunks at all
  const int i_chunks = (a.inter + kCols - 1) / kCols, s_chunks = (a.shared_inter + kCols - 1) / kCols;
  const auto begin2 = [&](Walk& w) {     // this warp's first chunk of expert w.j
    w.c = w.j < 0 ? warp : warp - sm->turn[w.j];
    if (w.c < 0) w.c += kMoeWarps;
  };
  const auto settle2 = [&](Walk& w) {    // on to the first chunk from w on that is this warp's
    while (w.c >= (w.j < 0 ? s_chunks : i_chunks)) {
      if (++w.j >= na) {
        w.j = j0;
        w.i += grid;
        if (w.i >= p.tiles3) return;
      }
      begin2(w);
    }
  };
  const auto first2 = [&]() {
    Walk w{cta, j0, 0};
    if (w.i < p.tiles3) {
      begin2(w);
      settle2(w);
    }
    return w;
  };
  const auto next2 = [&](Walk& w) {
    w.c += kMoeWarps;
    settle2(w);
  };

  // A stage: chunk c of `rows` rows from y0 on (and of as many from y1 on, when
  // y1 >= 0); K columns in all.
  int ls = 0;
  const auto load = [&](const CUtensorMap* m, const CUtensorMap* edge, int K, int c, int rows, int y0, int y1) {
    if (lane == 0) {
      uint64_t* full = &sm->full[warp][ls];
      const uint32_t dst = ring_a + ls * kStage;
      const int c0 = c * kCols, parts = y1 >= 0 ? 2 : 1;
      // whole blocks of 64 columns in one box; a chunk that holds the row's ragged
      // end takes a box per block, the last of which TMA fills with zeros
      if ((K & 63) == 0 || c0 + kCols <= (K & ~63)) {
        mbar_expect_tx(full, (uint32_t)(parts * rows * kCols * 2));
        tma3(dst, m, 0, y0, c0 >> 6, full);
        if (y1 >= 0) tma3(dst + kStage / 2, m, 0, y1, c0 >> 6, full);
      } else {
        const int nb = min((K - c0 + 63) >> 6, 2);
        mbar_expect_tx(full, (uint32_t)(parts * rows * nb * 128));
        for (int b = 0; b < nb; ++b) {
          tma2(dst + b * rows * 128, edge, c0 + b * 64, y0, full);
          if (y1 >= 0) tma2(dst + kStage / 2 + b * rows * 128, edge, c0 + b * 64, y1, full);
        }
      }
    }
    if (++ls == kStages) ls = 0;
  };
  int ahead = 0;                 // stages loaded and not yet multiplied
  Walk l1 = first1(), l2{0, 0, 0};
  int y1 = 0;                    // row of l1's tile, once the experts are chosen
  const auto row1 = [&]() {
    if (l1.i >= s_tiles && l1.i < n1) {
      const int j = (l1.i - s_tiles) / e_tiles;
      y1 = sm->expert[j] * 2 * a.inter + (l1.i - s_tiles - j * e_tiles) * 8;
    }
  };
  bool in2 = false;              // the loads have come to phase 2
  // Fills the stages that are free; before the choice only with the shared expert.
  const auto fill = [&](bool chosen) {
    while (ahead < kStages) {
      if (!in2) {
        if (any1 && l1.i < n1) {
          if (l1.i < s_tiles) {
            load(&maps.s_gate_up, &maps.s_gate_up_edge, a.hidden, l1.c, 8, 8 * l1.i, a.shared_inter + 8 * l1.i);
          } else {
            load(&maps.gate_up, &maps.gate_up_edge, a.hidden, l1.c, 8, y1, y1 + a.inter);
          }
          const int was = l1.i;
          next1(l1);
          if (l1.i != was) row1();
          ++ahead;
          continue;
        }
        if (!chosen) return;
        in2 = true;
        l2 = first2();
      }
      if (l2.i >= p.tiles3) return;
      if (l2.j < 0)
        load(&maps.s_down, &maps.s_down_edge, a.shared_inter, l2.c, p.rows3, l2.i * p.rows3, -1);
      else
        load(&maps.down, &maps.down_edge, a.inter, l2.c, p.rows3, sm->expert[l2.j] * a.hidden + l2.i * p.rows3, -1);
      next2(l2);
      ++ahead;
    }
  };
  fill(false);

  // ---- the choice of experts ----
  asm volatile("griddepcontrol.wait;" ::: "memory");   // kernel 1's logits
  if (!a.s_gate)
    for (int t = tid; t < a.tokens; t += kMoeThreads) sm->shared_w[t] = 1.0f;
  for (int t = warp; t < a.tokens; t += kMoeWarps) {
    if (a.experts <= 256) choose<8>(p, sm, t, lane);
    else if (a.experts <= 512) choose<16>(p, sm, t, lane);
    else choose<32>(p, sm, t, lane);
  }
  __syncthreads();
  build_lists(p, sm, tid);
  na = sm->n_active;
  n1 = s_tiles + na * e_tiles;
  row1();
  fill(true);

  const int g = lane >> 2, t4 = lane & 3;
  int cs = 0;
  uint32_t ph = 0;
  // The weights of 64 columns: row g in line `line` of the stage's 128-byte lines,
  // row g + 8 `up` bytes on.
  const auto weights = [&](Frag& f, int line, uint32_t up) {
    const uint8_t* at = ring + cs * kStage + line * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t off = (uint32_t)(((t4 + 4 * h) ^ (line & 7)) << 4);
      f.lo[h] = *reinterpret_cast<const uint4*>(at + off);
      f.hi[h] = *reinterpret_cast<const uint4*>(at + off + up);
    }
  };
  const auto done = [&]() {      // this stage is multiplied
    __syncwarp();
    if (++cs == kStages) {
      cs = 0;
      ph ^= 1u;
    }
    --ahead;
  };

  // ---- phase 1: act = weight silu(gate) up ----
  int flip = 0;
  for (int i = cta * kTeams + team; i < n1; i += tile_step) {
    const bool shared = i < s_tiles;
    const int j = shared ? -1 : (i - s_tiles) / e_tiles, r0 = (shared ? i : i - s_tiles - j * e_tiles) * 8;
    const int col0 = shared ? 0 : sm->base[j], cnt = shared ? a.tokens : sm->base[j + 1] - col0;
    const uint16_t* x[NG];       // the rows of this lane's columns
    float acc[NG][4];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const int c = 8 * n + g;
      const int cc = min(c, cnt - 1);   // columns past the expert's tokens repeat the last: never written
      x[n] = a.x + (size_t)(shared ? cc : sm->pair_t[col0 + cc]) * a.hidden + t4 * 8;
      acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
    }
    for (int c = member; c < h_chunks; c += kTeam) {
      uint4 b0[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) load_b(b0[h], x[0] + c * kCols + 64 * h, 0, a.hidden - c * kCols - 64 * h - t4 * 8, true);
      fill(true);                // the stage before's place, while these are on their way
      moe_wait(a, sm, &sm->full[warp][cs], ph);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (c * kCols + 64 * h >= a.hidden) break;
        Frag f;
        weights(f, h * 8 + g, kStage / 2);
        mma_block(acc[0], f, b0[h]);
#pragma unroll
        for (int n = 1; n < NG; ++n)
          if (8 * n < cnt) {
            uint4 b[2];
            load_b(b, x[n] + c * kCols + 64 * h, 0, a.hidden - c * kCols - 64 * h - t4 * 8, true);
            mma_block(acc[n], f, b);
          }
      }
      done();
    }
    // the team's four sums, in their order; lane (g, t4) of the first warp holds gate and
    // up of row g for columns 2 t4 and 2 t4 + 1
    const int cols = cols_of(j);
    uint16_t* const act = shared ? p.s_act : p.act;
    const size_t plane = (size_t)(shared ? a.tokens : a.tokens * a.top_k) * cols;
#pragma unroll
    for (int n = 0; n < NG; ++n)
      if (8 * n < cnt) {
        if (member > 0) sm->red[flip][warp][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        team_sync(team);
        if (member == 0) {
#pragma unroll
          for (int w = 1; w < kTeam; ++w) {
            const float4 v = sm->red[flip][warp + w][lane];
            acc[n][0] += v.x;
            acc[n][1] += v.y;
            acc[n][2] += v.z;
            acc[n][3] += v.w;
          }
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const int c = 8 * n + 2 * t4 + o;
            if (c < cnt) {
              const float v = silu(acc[n][o]) * acc[n][2 + o] * (shared ? sm->shared_w[c] : sm->pair_w[col0 + c]);
              const uint16_t hi = f32_to_bf16(v);
              const size_t at = (size_t)(col0 + c) * cols + r0 + g;
              act[at] = hi;
              act[plane + at] = f32_to_bf16(v - bf16_to_f32(hi));
            }
          }
        }
        flip ^= 1;
      }
  }

  // ---- every CTA's activations are there ----
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    atomicAdd(p.barrier, 1u);
    const long long t0 = clock64();
    while (true) {
      unsigned n;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(p.barrier) : "memory");
      if (n >= (unsigned)grid) break;
      if (clock64() - t0 > kBarrierBudget) {
        record_status(a.status, GDN_ERR_DEVICE_TIMEOUT);
        break;
      }
    }
    __threadfence();
  }
  __syncthreads();

  // ---- phase 2: y = sum over the experts of down act ----
  Walk w = first2();
  flip = 0;   // the teams met differently often
  for (int i = cta; i < p.tiles3; i += grid) {
    float acc[NG][4], low[NG][4];
#pragma unroll
    for (int n = 0; n < NG; ++n)
      acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = low[n][0] = low[n][1] = low[n][2] = low[n][3] = 0.0f;
    while (w.i == i) {
      const bool shared = w.j < 0;
      const int cols = cols_of(w.j), k = w.c * kCols + t4 * 8;
      uint32_t m0, m1;
      int base = 0;
      if (shared) {
        m0 = a.tokens < 32 ? (1u << a.tokens) - 1u : 0xffffffffu;
        m1 = a.tokens <= 32 ? 0u : (a.tokens < 64 ? (1u << (a.tokens - 32)) - 1u : 0xffffffffu);
      } else {
        const int e = sm->expert[w.j];
        m0 = sm->mask[e][0];
        m1 = sm->mask[e][1];
        base = sm->base[w.j];
      }
      const uint16_t* act = shared ? p.s_act : p.act;
      const size_t plane = (size_t)(shared ? a.tokens : a.tokens * a.top_k) * cols;
      bool have = false;
      Frag f[2];
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const uint32_t members = (n < 4 ? m0 >> (8 * n) : m1 >> (8 * n - 32)) & 0xffu;
        if (members == 0) continue;
        const int t = 8 * n + g;
        const bool use = members >> g & 1;
        const uint16_t* row = act + (size_t)(use ? (shared ? t : base + below(m0, m1, t)) : 0) * cols;
        uint4 hi[2][2], lo[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          load_b_cg(hi[h], row, k + 64 * h, cols, use);
          load_b_cg(lo[h], row + plane, k + 64 * h, cols, use);
        }
        if (!have) {
          fill(true);
          moe_wait(a, sm, &sm->full[warp][cs], ph);
          have = true;
#pragma unroll
          for (int h = 0; h < 2; ++h) weights(f[h], h * p.rows3 + g, 1024);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (w.c * kCols + 64 * h < cols) {
            mma_block(acc[n], f[h], hi[h]);
            mma_block(low[n], f[h], lo[h]);
          }
      }
      done();
      next2(w);
    }
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      if (8 * n >= a.tokens) break;
      sm->red[flip][warp][lane] =
          make_float4(acc[n][0] + low[n][0], acc[n][1] + low[n][1], acc[n][2] + low[n][2], acc[n][3] + low[n][3]);
      __syncthreads();
      const int r = tid & 15, t = 8 * n + (tid >> 4), h = i * p.rows3 + r;
      if (tid < 128 && t < a.tokens && r < p.rows3 && h < a.hidden) {
        const int l = (r & 7) * 4 + ((t & 7) >> 1);
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < kMoeWarps; ++q) {
          const float4 u = sm->red[flip][q][l];
          v += r < 8 ? (t & 1 ? u.y : u.x) : (t & 1 ? u.w : u.z);
        }
        const size_t at = (size_t)t * a.hidden + h;
        if (a.out_f32)
          static_cast<float*>(a.y)[at] = v;
        else
          static_cast<uint16_t*>(a.y)[at] = f32_to_bf16(v);
      }
      flip ^= 1;
    }
  }
}

PFN_cuTensorMapEncodeTiled_v12000 moe_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// Weights [rows][K]: boxes of 2 blocks of 64 columns by box_rows rows (of whole
// blocks), and boxes of one block (the ragged end of the rows included).
bool weight_maps(CUtensorMap* whole, CUtensorMap* edge, const void* base, uint64_t rows, uint64_t K, uint32_t box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = moe_encoder();
  if (!enc) return false;
  const cuuint32_t one[3] = {1, 1, 1};
  bool ok = true;
  if (K >= 64) {
    const cuuint64_t dims[3] = {64, rows, K / 64}, strides[2] = {K * 2, 128};
    const cuuint32_t box[3] = {64, box_rows, kCols / 64};
    ok = enc(whole, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  if (ok && K % 64 != 0) {
    const cuuint64_t dims[2] = {K, rows}, strides[1] = {K * 2};
    const cuuint32_t box[2] = {64, box_rows};
    ok = enc(edge, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  return ok;
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

template <int NG>
cudaError_t launch_experts(const MoeMaps& maps, const MoeParams& p, int grid, cudaStream_t stream) {
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(moe_experts_kernel<NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMoeSmem)) !=
      cudaSuccess)
    return e;
  // all CTAs wait for one another: a cooperative launch; it may begin while kernel 1
  // still runs
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeCooperative;
  at[0].val.cooperative = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kMoeThreads);
  cfg.dynamicSmemBytes = kMoeSmem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, moe_experts_kernel<NG>, maps, p);
}

}  // namespace

size_t moe_scratch_bytes(int tokens, int, int inter, int experts, int top_k, int shared_inter) {
  const size_t T = tokens > 0 ? tokens : 1;
  return 256 + up256(T * (experts + 1) * 8) + up256(T * top_k * inter * 4) + up256(T * shared_inter * 4);
}

cudaError_t launch_moe(const MoeArgs& a, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  MoeParams p;
  p.a = a;
  if (a.shared_inter == 0) p.a.s_gate = nullptr;
  const size_t T = a.tokens;
  char* ws = static_cast<char*>(a.scratch);
  p.barrier = reinterpret_cast<unsigned*>(ws);
  ws += 256;
  p.logit = reinterpret_cast<float2*>(ws);
  ws += up256(T * (a.experts + 1) * 8);
  p.act = reinterpret_cast<uint16_t*>(ws);
  ws += up256(T * a.top_k * a.inter * 4);
  p.s_act = reinterpret_cast<uint16_t*>(ws);
  // output rows: tiles of at most 16, as many as give every CTA the same number
  const int per = (a.hidden + 16 * sms - 1) / (16 * sms);
  p.rows3 = (a.hidden + per * sms - 1) / (per * sms);
  p.tiles3 = (a.hidden + p.rows3 - 1) / p.rows3;
  MoeMaps m;
  if (!weight_maps(&m.gate_up, &m.gate_up_edge, a.w_gate_up, (uint64_t)a.experts * 2 * a.inter, a.hidden, 8) ||
      !weight_maps(&m.down, &m.down_edge, a.w_down, (uint64_t)a.experts * a.hidden, a.inter, p.rows3))
    return cudaErrorInvalidValue;
  if (a.shared_inter > 0 &&
      (!weight_maps(&m.s_gate_up, &m.s_gate_up_edge, a.s_gate_up, 2ull * a.shared_inter, a.hidden, 8) ||
       !weight_maps(&m.s_down, &m.s_down_edge, a.s_down, a.hidden, a.shared_inter, p.rows3)))
    return cudaErrorInvalidValue;
  // one token: 2048 columns in flight per warp; more: 8 tokens share an expert's row
  const int rows = a.experts + (p.a.s_gate ? 1 : 0);
  if (a.tokens == 1)
    moe_router_kernel<1, 8><<<(rows + 7) / 8, 256, 0, stream>>>(p);
  else
    moe_router_kernel<8, 1><<<(rows * ((a.tokens + 7) / 8) + 7) / 8, 256, 0, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.tokens <= 8) return launch_experts<1>(m, p, sms, stream);
  if (a.tokens <= 16) return launch_experts<2>(m, p, sms, stream);
  if (a.tokens <= 32) return launch_experts<4>(m, p, sms, stream);
  return launch_experts<8>(m, p, sms, stream);
}

}  // namespace gdn
