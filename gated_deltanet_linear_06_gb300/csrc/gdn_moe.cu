// gdn_moe.cu -- a whole mixture-of-experts layer for a few tokens, in two
// kernels (HBM-bound: every chosen expert's weights are read once).
//
// Mathematics.  With few tokens each weight meets one or a few of them, so the
// layer costs its weights' bytes: 6 hidden inter per expert that any token
// chose.  The products run on the tensor cores all the same (m16n8k16: 16
// weight rows by 8 tokens), because their cost then does not grow with the
// tokens that share an expert.  Columns are tokens by their own number; a group
// of 8 tokens that an expert does not serve is skipped.
//
// Kernel 1, router logits: a warp per (expert, 8 tokens).  The chosen experts
// hang on which logits are larger, so the sums are compensated: each lane adds
// its products to S, which starts at a constant so large that it rounds them to
// a coarse grid exactly, and what S drops goes to a second sum; the two join in
// 64 bits.  Four operations a product, 4 us of 340 at 64 tokens.
//
// Kernel 2, one CTA per SM, everything else:
//   - a warp streams weights through a ring of 16 KB stages (16 rows x 512
//     columns by TMA, 128-byte swizzle): first the shared expert's, which need
//     no router and load while kernel 1 runs, then its share of the chosen
//     experts' gate and up rows, then of the down rows.  It runs ahead of the
//     products as far as the ring goes, past the grid barrier between the two
//     phases too: a step's down weights land while the last gate rows finish;
//   - eight warps choose the experts (every CTA for itself, which is cheaper
//     than another barrier), then multiply: warp w takes columns 64 w .. of each
//     stage, and the eight partial sums meet in shared memory in a fixed order.
//     Phase 1 tiles are 8 gate rows over the same 8 up rows, so silu(g) u forms
//     in one thread; the router's weight is multiplied in there.  Phase 2 tiles
//     are up to 16 output rows for ALL experts, so that a token's experts add up
//     in registers, in ascending order, without atomics or partial results.
// Nothing in a token's arithmetic depends on the other tokens.
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

constexpr int kMoeWarps = 8;                          // product warps
constexpr int kMoeThreads = 32 * (kMoeWarps + 1);
constexpr int kCols = 64 * kMoeWarps;                 // weight columns of a stage
constexpr uint32_t kStage = 16 * kCols * 2;
constexpr int kStages = 9;
constexpr int kMaxExperts = 1024, kMaxPairs = GDN_MOE_MAX_TOKENS * 32;
constexpr long long kBarrierBudget = 1LL << 31;       // clock cycles

struct MoeSmem {
  uint64_t full[kStages], empty[kStages], lists;
  int n_active;
  int gave_up;                         // a wait ran out: no later one waits
  int scan_a[kMoeWarps], scan_p[kMoeWarps];
  float4 red[2][kMoeWarps][32];
  uint32_t mask[kMaxExperts][2];       // tokens of an expert
  uint16_t expert[kMaxExperts];        // active experts, ascending
  uint16_t base[kMaxExperts];          // first pair of an active expert
  uint16_t rank[kMaxExperts];          // expert -> its place among the active
  float shared_w[GDN_MOE_MAX_TOKENS];  // the shared expert's factor
  uint16_t sel[kMaxPairs];             // chosen experts, token-major
  float sel_w[kMaxPairs];
  float pair_w[kMaxPairs];             // weights in the order of the pairs
};
constexpr uint32_t kMoeSmem = kStages * kStage + sizeof(MoeSmem) + 1024;
static_assert(kMoeSmem <= 227 * 1024, "shared memory");

struct MoeMaps {
  CUtensorMap gate_up, gate_up_edge, down, down_edge, s_gate_up, s_gate_up_edge, s_down, s_down_edge;
};

struct MoeParams {
  MoeArgs a;
  double* logit;        // [tokens][experts + 1]
  unsigned* barrier;    // arrivals of the grid barrier; zeroed by kernel 1
  uint16_t* act;        // [hi, lo][pairs][inter]
  uint16_t* s_act;      // [hi, lo][tokens][shared_inter]
  int rows3, tiles3;    // output rows per tile, tiles
};

// ---- kernel 1 ----
__global__ void __launch_bounds__(256) moe_router_kernel(const MoeParams p) {
  const MoeArgs& a = p.a;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.barrier = 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, unit = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int rows = a.experts + (a.s_gate ? 1 : 0), blocks = (a.tokens + 7) >> 3;
  if (unit >= rows * blocks) return;
  const int e = unit / blocks, t0 = (unit - e * blocks) * 8, nt = min(8, a.tokens - t0);
  const uint16_t* w = e < a.experts ? a.w_router + (size_t)e * a.hidden : a.s_gate;
  const uint16_t* x = a.x + (size_t)t0 * a.hidden;
  constexpr float kGrid = 3072.0f;   // products go to S on a grid of 2^-12
  float S[8], lo[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    S[t] = kGrid;
    lo[t] = 0.0f;
  }
  for (int k = lane * 8; k < a.hidden; k += 256) {
    const uint4 wv = __ldg(reinterpret_cast<const uint4*>(w + k));
    const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t >= nt) break;
      const uint4 xv = __ldg(reinterpret_cast<const uint4*>(x + (size_t)t * a.hidden + k));
      const uint32_t xx[4] = {xv.x, xv.y, xv.z, xv.w};
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
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    if (t >= nt) break;
    double v = (double)(S[t] - kGrid) + (double)lo[t];
    for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if (lane == 0) p.logit[(size_t)(t0 + t) * (a.experts + 1) + e] = v;
  }
}

// ---- kernel 2 ----

// e^x for x <= 0 given in 64 bits: the fp32 rounding of the argument is put
// back as a factor (at x = -80 it alone would cost 2^-18 of the result).
__device__ __forceinline__ float exp_of(double x) {
  const float h = (float)x;
  return h < -200.0f ? 0.0f : expf(h) * (1.0f + (float)(x - (double)h));
}

// A 64-bit key in the order of the doubles, NaN lowest.
__device__ __forceinline__ unsigned long long order_key(double v) {
  if (v != v) return 0;
  const long long b = __double_as_longlong(v + 0.0);   // -0 and 0 alike
  return (unsigned long long)(b ^ ((b >> 63) | (1ll << 63)));
}
__device__ __forceinline__ double order_value(unsigned long long k) {
  return __longlong_as_double((long long)(k ^ (k >> 63 ? 1ull << 63 : ~0ull)));
}

__device__ __forceinline__ void products_sync() {   // the product warps
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kMoeWarps) : "memory");
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

// Top-k of one token by one warp, into sel / sel_w.
__device__ void choose(const MoeParams& p, MoeSmem* sm, int t, int lane) {
  const MoeArgs& a = p.a;
  const double* lg = p.logit + (size_t)t * (a.experts + 1);
  unsigned long long key[kMaxExperts / 32];
  unsigned long long best = 0;
  int at = -1;
#pragma unroll
  for (int j = 0; j < kMaxExperts / 32; ++j) {
    if (j * 32 >= a.experts) break;
    const int e = j * 32 + lane;
    key[j] = e < a.experts ? order_key(__ldcg(lg + e)) : 0;
    if (e < a.experts && (at < 0 || key[j] > best)) {
      best = key[j];
      at = j;
    }
  }
  uint32_t used = 0;
  double top = 0.0;
  float den = 0.0f, sum = 0.0f, mine = 0.0f;
  for (int k = 0; k < a.top_k; ++k) {
    const uint32_t hi = at >= 0 ? (uint32_t)(best >> 32) : 0, mh = __reduce_max_sync(0xffffffffu, hi);
    const bool c1 = at >= 0 && hi == mh;
    const uint32_t lo = c1 ? (uint32_t)best : 0, ml = __reduce_max_sync(0xffffffffu, lo);
    const bool c2 = c1 && lo == ml;
    const int e = (int)__reduce_min_sync(0xffffffffu, c2 ? (uint32_t)(at * 32 + lane) : 0xffffffffu);
    const double v = order_value(((unsigned long long)mh << 32) | ml);
    if (k == 0) {   // the softmax's maximum and sum
      top = v;
#pragma unroll
      for (int j = 0; j < kMaxExperts / 32; ++j) {
        if (j * 32 >= a.experts) break;
        if (j * 32 + lane < a.experts) den += exp_of(order_value(key[j]) - top);
      }
      den = warp_sum(den);
    }
    const float w = exp_of(v - top);
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
      for (int j = 0; j < kMaxExperts / 32; ++j) {
        if (j * 32 >= a.experts) break;
        if (j * 32 + lane < a.experts && !(used >> j & 1) && (at < 0 || key[j] > best)) {
          best = key[j];
          at = j;
        }
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
  if (lane == 0 && a.s_gate) sm->shared_w[t] = sigmoid((float)__ldcg(lg + a.experts));
}

// The active experts in ascending order, their first pairs, and the pairs' weights.
__device__ void build_lists(const MoeParams& p, MoeSmem* sm, int tid) {
  const MoeArgs& a = p.a;
  const int warp = tid >> 5, lane = tid & 31;
  constexpr int PER = kMaxExperts / (32 * kMoeWarps);
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
  products_sync();
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
  if (tid == 0) sm->n_active = total;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    if (e < a.experts) {
      const int n = __popc(sm->mask[e][0]) + __popc(sm->mask[e][1]);
      if (n > 0) {
        sm->expert[ia] = (uint16_t)e;
        sm->base[ia] = (uint16_t)ip;
        sm->rank[e] = (uint16_t)ia;
        ++ia;
        ip += n;
      }
    }
  }
  products_sync();
  for (int i = tid; i < a.tokens * a.top_k; i += 32 * kMoeWarps) {
    const int t = i / a.top_k, e = sm->sel[i];
    const uint32_t below = t >= 32 ? 0xffffffffu : (1u << t) - 1u;
    const int r = __popc(sm->mask[e][0] & below) + (t >= 32 ? __popc(sm->mask[e][1] & ((1u << (t - 32)) - 1u)) : 0);
    sm->pair_w[sm->base[sm->rank[e]] + r] = sm->sel_w[i];
  }
  products_sync();
}

// Tokens of a mask below token t.
__device__ __forceinline__ int below(uint32_t m0, uint32_t m1, int t) {
  return t < 32 ? __popc(m0 & ((1u << t) - 1u)) : __popc(m0) + __popc(m1 & ((1u << (t - 32)) - 1u));
}

template <int NG>   // groups of 8 tokens
__global__ void __launch_bounds__(kMoeThreads, 1)
    moe_experts_kernel(const __grid_constant__ MoeMaps maps, const __grid_constant__ MoeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const MoeArgs& a = p.a;
  const uint32_t raw = tc::smem_u32(smem), pad = (1024u - (raw & 1023u)) & 1023u;
  uint8_t* const ring = smem + pad;
  MoeSmem* sm = reinterpret_cast<MoeSmem*>(ring + kStages * kStage);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x, grid = gridDim.x;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&sm->full[s], 1);
      tc::mbar_init(&sm->empty[s], kMoeWarps);
    }
    tc::mbar_init(&sm->lists, 1);
    sm->gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int e = tid; e < a.experts; e += kMoeThreads) sm->mask[e][0] = sm->mask[e][1] = 0;
  __syncthreads();

  const int s_tiles = a.shared_inter >> 3, e_tiles = a.inter >> 3;   // 8-row tiles of an expert
  int s = 0;
  uint32_t ph = 0;
  const auto step = [&]() {
    if (++s == kStages) {
      s = 0;
      ph ^= 1u;
    }
  };

  if (warp == kMoeWarps) {
    // ---- loads, by one thread ----
    if (lane == 0) {
      bool ok = true;
      const uint32_t ring_a = raw + pad;
      // One stage: columns c0 .. c0 + 511 of `rows` rows from y0 on (and of as many
      // from y1 on, when y1 >= 0); K columns in all.
      const auto load = [&](const CUtensorMap* m, const CUtensorMap* edge, int K, int c0, int rows, int y0, int y1) {
        ok = moe_wait(a, sm, &sm->empty[s], ph ^ 1u);
        if (!ok) return;
        const uint32_t dst = ring_a + s * kStage;
        const int parts = y1 >= 0 ? 2 : 1;
        // whole blocks of 64 columns in one box; a chunk that holds the row's ragged
        // end takes a box per block, the last of which TMA fills with zeros
        if ((K & 63) == 0 || c0 + kCols <= (K & ~63)) {
          mbar_expect_tx(&sm->full[s], (uint32_t)(parts * rows * kCols * 2));
          tma3(dst, m, 0, y0, c0 >> 6, &sm->full[s]);
          if (y1 >= 0) tma3(dst + kStage / 2, m, 0, y1, c0 >> 6, &sm->full[s]);
        } else {
          const int nb = (K - c0 + 63) >> 6;
          mbar_expect_tx(&sm->full[s], (uint32_t)(parts * rows * nb * 128));
          for (int b = 0; b < nb; ++b) {
            tma2(dst + b * rows * 128, edge, c0 + b * 64, y0, &sm->full[s]);
            if (y1 >= 0) tma2(dst + kStage / 2 + b * rows * 128, edge, c0 + b * 64, y1, &sm->full[s]);
          }
        }
        step();
      };
      for (int i = cta; i < s_tiles && ok; i += grid)
        for (int c0 = 0; c0 < a.hidden && ok; c0 += kCols)
          load(&maps.s_gate_up, &maps.s_gate_up_edge, a.hidden, c0, 8, 8 * i, a.shared_inter + 8 * i);
      if (ok) ok = moe_wait(a, sm, &sm->lists, 0);
      const int na = ok ? sm->n_active : 0, n1 = s_tiles + na * e_tiles;
      for (int i = cta + (s_tiles - cta + grid - 1 > 0 ? (s_tiles - cta + grid - 1) / grid * grid : 0); i < n1 && ok;
           i += grid) {
        const int j = (i - s_tiles) / e_tiles, r = (i - s_tiles - j * e_tiles) * 8;
        const int y = sm->expert[j] * 2 * a.inter + r;
        for (int c0 = 0; c0 < a.hidden && ok; c0 += kCols)
          load(&maps.gate_up, &maps.gate_up_edge, a.hidden, c0, 8, y, y + a.inter);
      }
      for (int i = cta; i < p.tiles3 && ok; i += grid) {
        for (int c0 = 0; c0 < a.shared_inter && ok; c0 += kCols)
          load(&maps.s_down, &maps.s_down_edge, a.shared_inter, c0, p.rows3, i * p.rows3, -1);
        for (int j = 0; j < na && ok; ++j)
          for (int c0 = 0; c0 < a.inter && ok; c0 += kCols)
            load(&maps.down, &maps.down_edge, a.inter, c0, p.rows3, sm->expert[j] * a.hidden + i * p.rows3, -1);
      }
    }
  } else {
    // ---- the choice of experts ----
    asm volatile("griddepcontrol.wait;" ::: "memory");   // kernel 1's logits
    if (!a.s_gate)
      for (int t = tid; t < a.tokens; t += 32 * kMoeWarps) sm->shared_w[t] = 1.0f;
    for (int t = warp; t < a.tokens; t += kMoeWarps) choose(p, sm, t, lane);
    products_sync();
    build_lists(p, sm, tid);
    if (tid == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(&sm->lists)) : "memory");
    const int na = sm->n_active, n1 = s_tiles + na * e_tiles;

    const int g = lane >> 2, t4 = lane & 3;
    int flip = 0;
    // this warp's 64 columns of the stage at hand: rows are `pitch` apart in the
    // order of the stage's 128-byte lines, the upper eight `up` bytes on
    const auto weights = [&](Frag& f, int line, uint32_t up) {
      const uint8_t* at = ring + s * kStage + line * 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t off = (uint32_t)(((t4 + 4 * h) ^ (line & 7)) << 4);
        f.lo[h] = *reinterpret_cast<const uint4*>(at + off);
        f.hi[h] = *reinterpret_cast<const uint4*>(at + off + up);
      }
    };
    const auto release = [&]() {
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(&sm->empty[s])) : "memory");
      step();
    };

    // ---- phase 1: act = weight silu(gate) up ----
    for (int i = cta; i < n1; i += grid) {
      const bool shared = i < s_tiles;
      const int j = shared ? 0 : (i - s_tiles) / e_tiles, r0 = (shared ? i : i - s_tiles - j * e_tiles) * 8;
      uint32_t m0 = 0xffffffffu, m1 = 0xffffffffu;
      if (!shared) {
        const int e = sm->expert[j];
        m0 = sm->mask[e][0];
        m1 = sm->mask[e][1];
      }
      float acc[NG][4];
      uint32_t groups = 0;
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        if ((n < 4 ? m0 >> (8 * n) : m1 >> (8 * n - 32)) & 0xffu) groups |= 1u << n;
        if (8 * n >= a.tokens) groups &= ~(1u << n);
        acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
      }
      for (int c0 = 0; c0 < a.hidden; c0 += kCols) {
        const int k = c0 + warp * 64 + t4 * 8;
        const bool in = c0 + warp * 64 < a.hidden;
        uint4 b[2];
        int first = __ffs(groups) - 1;
        if (in) load_b(b, a.x + (size_t)(8 * first + g) * a.hidden, k, a.hidden, 8 * first + g < a.tokens);
        moe_wait(a, sm, &sm->full[s], ph);
        if (in) {
          Frag f;
          weights(f, warp * 8 + g, kStage / 2);
#pragma unroll
          for (int n = 0; n < NG; ++n)
            if (groups >> n & 1) {
              if (n != first)
                load_b(b, a.x + (size_t)(8 * n + g) * a.hidden, k, a.hidden, 8 * n + g < a.tokens);
              mma_block(acc[n], f, b);
            }
        }
        release();
      }
      const int cols = shared ? a.shared_inter : a.inter;
      uint16_t* const act = shared ? p.s_act : p.act;
      const size_t plane = (size_t)(shared ? a.tokens : a.tokens * a.top_k) * cols;
#pragma unroll
      for (int n = 0; n < NG; ++n)
        if (groups >> n & 1) {
          sm->red[flip][warp][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
          products_sync();
          const int r = tid & 7, t = 8 * n + (tid >> 3);
          if (tid < 64 && t < a.tokens && ((t < 32 ? m0 >> t : m1 >> (t - 32)) & 1)) {
            const int l = r * 4 + ((t & 7) >> 1), o = t & 1;
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < kMoeWarps; ++w) {
              const float4 v = sm->red[flip][w][l];
              gate += o ? v.y : v.x;
              up += o ? v.w : v.z;
            }
            const int pair = shared ? t : sm->base[j] + below(m0, m1, t);
            const float v = silu(gate) * up * (shared ? sm->shared_w[t] : sm->pair_w[pair]);
            const uint16_t hi = f32_to_bf16(v);
            const size_t at = (size_t)pair * cols + r0 + r;
            act[at] = hi;
            act[plane + at] = f32_to_bf16(v - bf16_to_f32(hi));
          }
          flip ^= 1;
        }
    }

    // ---- every CTA's activations are there ----
    __threadfence();
    products_sync();
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
    products_sync();

    // ---- phase 2: y = sum over the experts of down act ----
    for (int i = cta; i < p.tiles3; i += grid) {
      float acc[NG][4];
#pragma unroll
      for (int n = 0; n < NG; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
      for (int j = a.shared_inter > 0 ? -1 : 0; j < na; ++j) {
        const bool shared = j < 0;
        const int cols = shared ? a.shared_inter : a.inter;
        const uint16_t* act = shared ? p.s_act : p.act;
        const size_t plane = (size_t)(shared ? a.tokens : a.tokens * a.top_k) * cols;
        uint32_t m0 = 0xffffffffu, m1 = 0xffffffffu;
        int base = 0;
        if (!shared) {
          const int e = sm->expert[j];
          m0 = sm->mask[e][0];
          m1 = sm->mask[e][1];
          base = sm->base[j];
        }
        for (int c0 = 0; c0 < cols; c0 += kCols) {
          const int k = c0 + warp * 64 + t4 * 8;
          const bool in = c0 + warp * 64 < cols;
          bool have = false;
          Frag f;
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            const uint32_t members = (n < 4 ? m0 >> (8 * n) : m1 >> (8 * n - 32)) & 0xffu;
            if (members == 0 || 8 * n >= a.tokens) continue;
            const int t = 8 * n + g;
            const bool use = t < a.tokens && (members >> g & 1);
            const uint16_t* row = act + (size_t)(shared ? (use ? t : 0) : base + (use ? below(m0, m1, t) : 0)) * cols;
            uint4 hi[2], lo[2];
            if (in) {
              load_b_cg(hi, row, k, cols, use);
              load_b_cg(lo, row + plane, k, cols, use);
            }
            if (!have) {
              moe_wait(a, sm, &sm->full[s], ph);
              have = true;
              if (in) weights(f, warp * p.rows3 + g, 1024);
            }
            if (in) {
              mma_block(acc[n], f, hi);
              mma_block(acc[n], f, lo);
            }
          }
          release();
        }
      }
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        if (8 * n >= a.tokens) break;
        sm->red[flip][warp][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        products_sync();
        const int r = tid & 15, t = 8 * n + (tid >> 4), h = i * p.rows3 + r;
        if (tid < 128 && t < a.tokens && r < p.rows3 && h < a.hidden) {
          const int l = (r & 7) * 4 + ((t & 7) >> 1);
          float v = 0.0f;
#pragma unroll
          for (int w = 0; w < kMoeWarps; ++w) {
            const float4 q = sm->red[flip][w][l];
            v += r < 8 ? (t & 1 ? q.y : q.x) : (t & 1 ? q.w : q.z);
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

// Weights [rows][K]: boxes of 8 blocks of 64 columns by box_rows rows (of whole
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
  p.logit = reinterpret_cast<double*>(ws);
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
  const int units = (a.experts + (p.a.s_gate ? 1 : 0)) * ((a.tokens + 7) / 8);
  moe_router_kernel<<<(units + 7) / 8, 256, 0, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.tokens <= 8) return launch_experts<1>(m, p, sms, stream);
  if (a.tokens <= 16) return launch_experts<2>(m, p, sms, stream);
  if (a.tokens <= 32) return launch_experts<4>(m, p, sms, stream);
  return launch_experts<8>(m, p, sms, stream);
}

}  // namespace gdn
