// gdn_moe.cu -- a whole mixture-of-experts layer for a few tokens (HBM-bound:
// every chosen expert's weights are read once).
//
// Mathematics.  With few tokens each weight meets one or a few of them, so the
// layer costs its weights' bytes: 6 hidden inter per expert that any token
// chose.  The products run on the tensor cores all the same (m16n8k16: 16
// weight rows by 8 tokens), because their cost then does not grow with the
// tokens that share an expert.
//
// Four launches by programmatic dependent launch, each begun while the one before it
// runs (the first: as the caller's last ends), so that between them only data is
// waited for:
//   router   logits: a CTA takes 8 experts and 8 tokens, one warp an expert.  The
//            chosen experts hang on which logits are larger, so the sums are
//            compensated: the products are exact in fp32, a lane adds them to two
//            sums S and what each addition drops (Knuth's two-sum) to a second
//            sum beside each.  With n products a sum the error is below
//            ((n + 6) 2^-24)^2 of the products' sizes, whatever their scale, and
//            some 2^-45 as a rule.  (S on a grid fixed for logits of size 1 cost 4
//            operations a product where this costs 7, of which fp32 pairs do two at
//            once (64 tokens 21 us for 26.5, 16 tokens 8 for 9.5), but kept no more
//            than fp32 for activations of 1e-4 and sums beyond 2^10.)  Logits stay
//            pairs of fp32 from there on (fp64 additions run at 1/64 of the rate here:
//            with them the choice of 8 experts alone took 12 us).
//   choice   a CTA per token: a bound from the lanes' maxima, then the few
//            candidates above it count those before them (a warp that picked one
//            maximum after the other took 15 us per token with 512 experts).
//   gate_up  tiles of 8 gate rows over the same 8 up rows, so that silu(g) u forms
//            in one thread; columns are the expert's own tokens; four warps share
//            a tile, each with every fourth chunk of 128 weight columns.
//   down     up to 16 output rows per CTA for ALL experts, so that a token's
//            experts add up on the SM without atomics or partial results: columns
//            are the expert's own tokens, a chunk's product is added to the warp's
//            own [token][row] sums in shared memory, and the warps' sums meet at
//            the end.  (With all tokens as columns and the sums in registers, 64
//            tokens took 40 % more instructions.)
// In the last two every warp feeds itself: it has two stages of 4 KB (16 rows x
// 128 columns, by TMA, 128-byte swizzle) and refills a stage once it has
// multiplied it, so 16 warps keep some 100 KB on their way and no warp waits for
// another's data.  The shared expert's weights load before the choice is made,
// and a CTA's first down weights before the last gate rows of others are done.
// (Measured on the way: stages multiplied by 8 or 16 warps together cost the
// latency of their activations and the warps' meetings, 1500 clocks where the
// bytes take 700; all phases in one cooperative kernel lost 4 us before its
// start, for the runtime lets such a launch begin only after the one before.)
// Which warp adds what depends on the expert's and the chunk's numbers alone, so
// nothing in a token's arithmetic depends on the other tokens.
//
// Measured, all four (hidden 2048; router, choice, gate_up, down apart in us): one
// token through 8 of 256 experts of 512 22.4 us (4, 5, 11, 10, overlapped); 16 tokens
// 117 (10, 5, 65, 45); 64 tokens through 10 of 512 experts 415 (27, 6, 260, 135),
// 5.6 TB/s or 82 % of a copy's rate; 5 tokens through 6 of 64 experts of 1408 with an
// fp32 result 89 to 95 (9, 4, 47, 43).  gate_up runs at the memory's rate.  down's warps
// are bound by their instructions (some 400 a chunk), and few experts spread unevenly over the four
// teams (21 to 32 chunks a warp at 16 tokens).  A team's four warps take every fourth
// chunk of 128 columns: experts of 512 keep all of them busy alike, of 128 or 256 one or
// two of four, of 768 two twice as long as the others.
//
// The activations between the products are kept as sums of bf16, because the
// tensor cores take both operands in one 16-bit type: two (16 bits of
// significand) for a bf16 output, where one would cost 2^-9 of each, and three
// (24 bits) for an fp32 output.  The products on the low parts cost tensor time,
// not bytes.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_launch.h"
#include "gdn_prefill.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kTeam = 4, kTeams = 4, kMoeWarps = kTeam * kTeams, kMoeThreads = 32 * kMoeWarps;
constexpr int kCols = 128;                            // weight columns of a stage
constexpr uint32_t kStage = 16 * kCols * 2;
constexpr int kStages = 2;                            // of each warp
constexpr uint32_t kRing = kMoeWarps * kStages * kStage;
constexpr int kMaxExperts = 1024, kMaxPairs = GDN_MOE_MAX_TOKENS * 32;
constexpr int kRouterCols = 2048, kRouterWarps = 8;
constexpr uint32_t kRouterSmem = 16 * kRouterCols * 2;
constexpr int kChoiceThreads = 256;

// What the choice leaves to the products, in the workspace, token-major.
struct Choice {
  float shared_w[GDN_MOE_MAX_TOKENS];  // the shared expert's factors
  float weight[kMaxPairs];
  uint16_t expert[kMaxPairs];
};

// The active experts, ascending, and their tokens: each CTA of the products makes
// them for itself.
struct Lists {
  int n_active, n_team[kTeams];
  int scan_a[kMoeWarps], scan_p[kMoeWarps];
  uint32_t mask[kMaxExperts][2];       // tokens, first of an expert, then of an active one
  uint16_t expert[kMaxExperts];        // active experts
  uint16_t base[kMaxExperts + 8];      // their first pairs
  uint16_t rank[kMaxExperts];          // expert -> its place among the active
  uint8_t pair_t[kMaxPairs];           // tokens of the (expert, token) pairs
  union {
    float pair_w[kMaxPairs];                 // gate_up: and their weights
    uint32_t of_team[kTeams][kMaxExperts / kTeams];   // down: the active experts e = team (mod kTeams), as Entry
  };
};

// An expert and its pairs in one word: number, first pair, pairs.
struct Entry {
  static constexpr uint32_t kShared = 1u << 31;   // the shared expert: all tokens, in order
  static __device__ __forceinline__ uint32_t of(int e, int base, int cnt) {
    return (uint32_t)e | (uint32_t)base << 10 | (uint32_t)cnt << 21;
  }
  static __device__ __forceinline__ int expert(uint32_t v) { return v & 1023; }
  static __device__ __forceinline__ int base(uint32_t v) { return v >> 10 & 2047; }
  static __device__ __forceinline__ int count(uint32_t v) { return v >> 21 & 127; }
  static __device__ __forceinline__ bool shared(uint32_t v) { return (int32_t)v < 0; }
};
static_assert(kMaxExperts <= 1024 && kMaxPairs <= 2048 && GDN_MOE_MAX_TOKENS < 128, "an entry's fields");

struct MoeMaps {
  CUtensorMap whole, edge, s_whole, s_edge;   // of the experts, of the shared expert
};

struct MoeParams {
  MoeArgs a;
  float2* logit;        // [tokens][experts + 1], high and low part
  Choice* choice;
  uint16_t* act;        // [part][pairs][inter]; two parts, or three
  uint16_t* s_act;      // [part][tokens][shared_inter]
  int rows3, tiles3;    // output rows per tile, tiles
};

__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// a + b as a rounded sum and its error (Knuth's two-sum).
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float s = a + b, bb = s - a;
  return make_float2(s, (a - (s - bb)) + (b - bb));
}

__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// S += x w, and what the sum's rounding drops to lo: two two-sums of S and the exact
// product x w, in pairs.
__device__ __forceinline__ void add_product(float2& S, float2& lo, float2 x, float2 w) {
  const float2 minus = make_float2(-1.0f, -1.0f);
  const float2 s = __ffma2_rn(x, w, S);
  const float2 nb = __ffma2_rn(s, minus, S);                       // -(s - S), what s took of x w
  const float2 of_S = __ffma2_rn(__fadd2_rn(s, nb), minus, S);     // what s dropped of S
  const float2 of_xw = __ffma2_rn(x, w, nb);                       // ... and of x w
  lo = __fadd2_rn(lo, __fadd2_rn(of_S, of_xw));
  S = s;
}

// One wait of a warp, all its lanes alike (they meet again right after it).  After a
// wait that gave up the results are unspecified; the status word tells.
__device__ __forceinline__ bool moe_wait(const MoeArgs& a, uint64_t* mbar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred P1;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 P1, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, P1;\n\t}\n"
      : "=r"(done)
      : "r"(tc::smem_u32(mbar)), "r"(parity)
      : "memory");
  if (__all_sync(0xffffffffu, done)) return true;
  if (__all_sync(0xffffffffu, tc::mbar_wait(mbar, parity, kWaitBudget))) return true;
  record_status(a.status, GDN_ERR_DEVICE_TIMEOUT);
  return false;
}

// ---- router ----
template <int NT>   // tokens of a CTA
__global__ void __launch_bounds__(32 * kRouterWarps) moe_router_kernel(const MoeParams p) {
  extern __shared__ __align__(128) uint8_t rows_raw[];
  __shared__ __align__(8) uint64_t full;
  uint16_t* const rows = reinterpret_cast<uint16_t*>(rows_raw);   // 8 experts, 8 tokens
  const MoeArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_rows = a.experts + (a.s_gate ? 1 : 0);
  const int e0 = blockIdx.x * 8, t0 = blockIdx.y * NT, ne = min(8, n_rows - e0), nt = min(NT, a.tokens - t0);
  if (threadIdx.x == 0) {
    tc::mbar_init(&full, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  // The kernel before this call is done; only then may the next begin, for the products
  // load weights before they wait.
  wait_before();
  let_next_begin();
  float2 S[NT], lo[NT];   // of even and of odd columns
#pragma unroll
  for (int t = 0; t < NT; ++t) S[t] = lo[t] = make_float2(0.0f, 0.0f);
  bool ok = true;
  uint32_t ph = 0;
  for (int k0 = 0; k0 < a.hidden; k0 += kRouterCols, ph ^= 1u) {
    const int n = min(kRouterCols, a.hidden - k0);
    if (warp == 0 && ok) {   // a row per lane
      if (lane == 0) mbar_expect_tx(&full, (uint32_t)((ne + nt) * n * 2));
      __syncwarp();
      if (lane < ne + nt) {
        const bool is_x = lane >= ne;
        const int r = is_x ? lane - ne : e0 + lane;
        const uint16_t* src = is_x ? a.x + (size_t)(t0 + r) * a.hidden
                                   : (r < a.experts ? a.w_router + (size_t)r * a.hidden : a.s_gate);
        bulk_copy(rows + (is_x ? 8 + r : lane) * kRouterCols, src + k0, (uint32_t)n * 2, &full);
      }
    }
    ok = ok && moe_wait(a, &full, ph);
    if (ok && warp < ne) {
      for (int k = lane * 8; k < n; k += 256) {
        const uint4 wv = *reinterpret_cast<const uint4*>(rows + warp * kRouterCols + k);
        const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int t = 0; t < NT; ++t) {   // past the end the last token again
          const uint4 xv = *reinterpret_cast<const uint4*>(rows + (8 + min(t, nt - 1)) * kRouterCols + k);
          const uint32_t xx[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) add_product(S[t], lo[t], bf16_pair(xx[i]), bf16_pair(ww[i]));
        }
      }
    }
    __syncthreads();   // the rows' places are free
  }
  if (warp >= ne) return;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    // the sums (S, lo) join as pairs: the high parts' rounding is kept
    const float2 both = two_sum(S[t].x, S[t].y);
    float h = both.x, l = (lo[t].x + lo[t].y) + both.y;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
      const float oh = __shfl_xor_sync(0xffffffffu, h, m), ol = __shfl_xor_sync(0xffffffffu, l, m);
      const float2 r = two_sum(h, oh);
      h = r.x;
      l = (l + ol) + r.y;
    }
    // (an infinite or NaN sum has no remainder: what was dropped on the way is NaN then)
    if (lane == 0 && t < nt)
      p.logit[(size_t)(t0 + t) * (a.experts + 1) + e0 + warp] = isfinite(h) ? two_sum(h, l) : make_float2(h, 0.0f);
  }
}

// ---- choice ----

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

// Tokens of a mask below token t.
__device__ __forceinline__ int below(uint32_t m0, uint32_t m1, int t) {
  return t < 32 ? __popc(m0 & ((1u << t) - 1u)) : __popc(m0) + __popc(m1 & ((1u << (t - 32)) - 1u));
}

// One token.  Of the 32 lanes' maxima the k-th largest bounds the k-th largest key
// from below, so only keys from there on (some k of them) are candidates; a
// candidate's rank is the number of candidates with a larger key, or an equal one
// and a lower index.  Ranks below top_k are the choice, in order.
__global__ void __launch_bounds__(kChoiceThreads) moe_choice_kernel(const MoeParams p) {
  __shared__ unsigned long long key[kMaxExperts];
  __shared__ uint16_t cand[kMaxExperts];
  __shared__ int n_cand;
  __shared__ float part[kChoiceThreads / 32];
  __shared__ float chosen[32];
  const MoeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, t = blockIdx.x;
  let_next_begin();
  if (tid == 0) n_cand = 0;
  wait_before();   // the logits
  const float2* lg = p.logit + (size_t)t * (a.experts + 1);
  for (int e = tid; e < a.experts; e += kChoiceThreads) key[e] = order_key(__ldcg(lg + e));
  __syncthreads();
  // every warp: the lanes' maxima, the softmax's maximum, the bound
  unsigned long long m = 0;
  for (int e = lane; e < a.experts; e += 32) m = max(m, key[e]);
  const uint32_t mine = (uint32_t)(m >> 32), h = __reduce_max_sync(0xffffffffu, mine);
  const uint32_t l = __reduce_max_sync(0xffffffffu, mine == h ? (uint32_t)m : 0u);
  const float2 top = order_value(((unsigned long long)h << 32) | l);
  int above = 0;
  for (int o = 0; o < 32; ++o) {
    const uint32_t v = __shfl_sync(0xffffffffu, mine, o);
    above += v > mine || (v == mine && o < lane);
  }
  const uint32_t bound = __reduce_max_sync(0xffffffffu, above == a.top_k - 1 ? mine : 0u);
  float den = 0.0f;
  for (int e = tid; e < a.experts; e += kChoiceThreads) {
    const unsigned long long k = key[e];
    den += exp_of(order_value(k), top);
    if ((uint32_t)(k >> 32) >= bound) cand[atomicAdd(&n_cand, 1)] = (uint16_t)e;
  }
  den = warp_sum(den);
  if (lane == 0) part[tid >> 5] = den;
  __syncthreads();
  const int n = n_cand;
  for (int i = tid; i < n; i += kChoiceThreads) {
    const int e = cand[i];
    const unsigned long long k = key[e];
    int rank = 0;
    for (int o = 0; o < n; ++o) {
      const int f = cand[o];
      rank += key[f] > k || (key[f] == k && f < e);
    }
    if (rank < a.top_k) {
      chosen[rank] = exp_of(order_value(k), top);
      p.choice->expert[t * a.top_k + rank] = (uint16_t)e;
      if (a.topk_id) a.topk_id[t * a.top_k + rank] = e;
    }
  }
  __syncthreads();
  if (tid < 32) {
    float sum = 0.0f;   // in the order of the warps, or of the ranks
    for (int w = 0; w < kChoiceThreads / 32; ++w) sum += part[w];
    if (a.renorm && sum == sum) {   // with a NaN among the logits all of the softmax is NaN
      sum = 0.0f;
      for (int k = 0; k < a.top_k; ++k) sum += chosen[k];
    }
    if (lane < a.top_k) {
      const float w = chosen[lane] / sum;
      p.choice->weight[t * a.top_k + lane] = w;
      if (a.topk_w) a.topk_w[t * a.top_k + lane] = w;
    }
    if (lane == 0) p.choice->shared_w[t] = a.s_gate ? sigmoid(__ldcg(lg + a.experts).x) : 1.0f;
  }
}

// ---- products ----

// The teams' experts, a warp per team.
__device__ __forceinline__ void team_lists(Lists& L, int warp, int lane) {
  if (warp >= kTeams) return;
  int n = 0;
  for (int j = lane; j - lane < L.n_active; j += 32) {
    const bool in = j < L.n_active && L.expert[j] % kTeams == warp;
    const uint32_t b = __ballot_sync(0xffffffffu, in);
    if (in)
      L.of_team[warp][n + __popc(b & ((1u << lane) - 1u))] =
          Entry::of(L.expert[j], L.base[j], L.base[j + 1] - L.base[j]);
    n += __popc(b);
  }
  if (lane == 0) L.n_team[warp] = n;
}

// The lists, by all threads of a CTA, with the pairs' weights or the teams' experts.
template <bool weights>
__device__ __forceinline__ void make_lists(const MoeParams& p, Lists& L) {
  const MoeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = a.tokens * a.top_k;
  if (a.tokens == 1) {   // the choice, sorted (1 us less than by the way of all experts)
    if (tid < n) {
      const int e = __ldcg(&p.choice->expert[tid]);
      int r = 0;
      for (int o = 0; o < n; ++o) r += __shfl_sync(__activemask(), e, o) < e;
      L.expert[r] = (uint16_t)e;
      L.base[r] = (uint16_t)r;
      L.pair_t[r] = 0;
      if (weights) L.pair_w[r] = __ldcg(&p.choice->weight[tid]);
    }
    if (tid == 0) {
      L.n_active = n;
      L.base[n] = (uint16_t)n;
    }
    __syncthreads();
    if (!weights) team_lists(L, warp, lane);
    __syncthreads();
    return;
  }
  for (int e = tid; e < a.experts; e += kMoeThreads) L.mask[e][0] = L.mask[e][1] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kMoeThreads) {
    const int t = i / a.top_k;
    atomicOr(&L.mask[__ldcg(&p.choice->expert[i])][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  constexpr int PER = (kMaxExperts + kMoeThreads - 1) / kMoeThreads;
  uint32_t m0[PER], m1[PER];
  int na = 0, np = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    m0[i] = e < a.experts ? L.mask[e][0] : 0;
    m1[i] = e < a.experts ? L.mask[e][1] : 0;
    na += (m0[i] | m1[i]) != 0;
    np += __popc(m0[i]) + __popc(m1[i]);
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
    L.scan_a[warp] = ia;
    L.scan_p[warp] = ip;
  }
  __syncthreads();   // (and every mask is in registers)
  ia -= na;
  ip -= np;
  for (int w = 0; w < kMoeWarps; ++w)
    if (w < warp) {
      ia += L.scan_a[w];
      ip += L.scan_p[w];
    }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if ((m0[i] | m1[i]) != 0) {
      const int e = tid * PER + i;
      L.expert[ia] = (uint16_t)e;
      L.base[ia] = (uint16_t)ip;
      L.mask[ia][0] = m0[i];
      L.mask[ia][1] = m1[i];
      L.rank[e] = (uint16_t)ia;
      ++ia;
      ip += __popc(m0[i]) + __popc(m1[i]);
    }
  if (tid == kMoeThreads - 1) {
    L.n_active = ia;
    L.base[ia] = (uint16_t)ip;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kMoeThreads) {
    const int t = i / a.top_k, j = L.rank[__ldcg(&p.choice->expert[i])];
    const int at = L.base[j] + below(L.mask[j][0], L.mask[j][1], t);
    if (weights) L.pair_w[at] = __ldcg(&p.choice->weight[i]);
    L.pair_t[at] = (uint8_t)t;
  }
  if (!weights) team_lists(L, warp, lane);
  __syncthreads();
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

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 rows x 64 columns of weights by 8 tokens.  Each lane holds 8 columns in a
// row of A and of B, 16 bytes each, so that the columns of the four products
// are those of four lanes: a permutation of the columns, the same in both.
struct Frag {
  uint4 lo[2], hi[2];   // row g and row g + 8, column halves
};
__device__ __forceinline__ void mma_block(float (&c)[4], const Frag& f, const uint4* b) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    mma16816(c, f.lo[h].x, f.hi[h].x, f.lo[h].y, f.hi[h].y, b[h].x, b[h].y);
    mma16816(c, f.lo[h].z, f.hi[h].z, f.lo[h].w, f.hi[h].w, b[h].z, b[h].w);
  }
}

// A warp's stage: chunk c of `rows` rows from y0 on (and of as many from y1 on,
// when y1 >= 0); K columns in all.  By one lane.  Whole blocks of 64 columns come
// in one box; a chunk that holds the row's ragged end takes a box per block, the
// last of which TMA fills with zeros.
__device__ __noinline__ void load_ragged(uint32_t dst, uint64_t* full, const CUtensorMap* edge, int K, int c, int rows,
                                         int y0, int y1) {
  const int c0 = c * kCols, parts = y1 >= 0 ? 2 : 1, nb = min((K - c0 + 63) >> 6, 2);
  mbar_expect_tx(full, (uint32_t)(parts * rows * nb * 128));
  for (int b = 0; b < nb; ++b) {
    tma2(dst + b * rows * 128, edge, c0 + b * 64, y0, full);
    if (y1 >= 0) tma2(dst + kStage / 2 + b * rows * 128, edge, c0 + b * 64, y1, full);
  }
}
template <bool two>
__device__ __forceinline__ void load_stage(uint32_t dst, uint64_t* full, const CUtensorMap* whole,
                                           const CUtensorMap* edge, int K, int c, int rows, int y0, int y1) {
  if ((K & 63) == 0 || (c + 1) * kCols <= (K & ~63)) {
    mbar_expect_tx(full, (uint32_t)((two ? 2 : 1) * rows * kCols * 2));
    tma3(dst, whole, 0, y0, c * (kCols / 64), full);
    if (two) tma3(dst + kStage / 2, whole, 0, y1, c * (kCols / 64), full);
  } else {
    load_ragged(dst, full, edge, K, c, rows, y0, two ? y1 : -1);
  }
}

// The weights of 64 columns: row g in line `line` of the stage's 128-byte lines,
// row g + 8 `up` bytes on.
__device__ __forceinline__ void load_a(Frag& f, const uint8_t* stage, int line, uint32_t up, int t4) {
  const uint8_t* at = stage + line * 128;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t off = (uint32_t)(((t4 + 4 * h) ^ (line & 7)) << 4);
    f.lo[h] = *reinterpret_cast<const uint4*>(at + off);
    f.hi[h] = *reinterpret_cast<const uint4*>(at + off + up);
  }
}

struct ProductSmem {
  uint64_t full[kMoeWarps][kStages];
  Lists lists;
  float4 red[2][kMoeWarps][32];        // gate_up; in its place down's sums
};
constexpr uint32_t kGateUpSmem = kRing + sizeof(ProductSmem) + 1024;
constexpr int kSumRow = 17;            // a token's 16 sums, and one to spread the banks
constexpr uint32_t down_smem(int tokens) {
  return kRing + offsetof(ProductSmem, red) + kMoeWarps * tokens * kSumRow * 4 + 1024;
}
static_assert(kGateUpSmem <= 227 * 1024 && down_smem(GDN_MOE_MAX_TOKENS) <= 227 * 1024, "shared memory");

template <int NG>   // groups of 8 tokens
__global__ void __launch_bounds__(kMoeThreads, 1)
    moe_gate_up_kernel(const __grid_constant__ MoeMaps maps, const __grid_constant__ MoeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const MoeArgs& a = p.a;
  const uint32_t raw = tc::smem_u32(smem), pad = (1024u - (raw & 1023u)) & 1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x, grid = gridDim.x;
  const int team = warp / kTeam, member = warp % kTeam;
  ProductSmem* sm = reinterpret_cast<ProductSmem*>(smem + pad + kRing);
  uint8_t* const ring = smem + pad + warp * kStages * kStage;          // this warp's
  const uint32_t ring_a = raw + pad + warp * kStages * kStage;
  uint64_t* const full = sm->full[warp];
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) tc::mbar_init(&full[s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  const int s_tiles = a.shared_inter >> 3, e_tiles = a.inter >> 3;   // 8-row tiles of an expert
  const int h_chunks = (a.hidden + kCols - 1) / kCols, tile_step = grid * kTeams;
  const int i0 = cta * kTeams + team;
  int n_tiles = s_tiles;
  // the loads' place: tile, chunk, the tile's rows; free stages
  int li = member < h_chunks ? i0 : 0x7fffffff, lc = member, ly = 8 * i0, ls = 0, free_stages = kStages;
  // After a wait that gave up no later one waits and nothing more is asked for (a stage
  // whose copy is late is still armed); what is on its way had that wait to arrive in.
  bool ok = true;
  const auto fill = [&]() {
    while (ok && free_stages > 0 && li < n_tiles) {
      const bool shared = li < s_tiles;
      if (lane == 0)
        load_stage<true>(ring_a + ls * kStage, &full[ls], shared ? &maps.s_whole : &maps.whole,
                   shared ? &maps.s_edge : &maps.edge, a.hidden, lc, 8, ly, ly + (shared ? a.shared_inter : a.inter));
      __syncwarp();
      --free_stages;
      if (++ls == kStages) ls = 0;
      lc += kTeam;
      if (lc >= h_chunks) {
        lc = member;
        li += tile_step;
        ly = 8 * li;
        if (li >= s_tiles && li < n_tiles) {
          const int j = (li - s_tiles) / e_tiles;
          ly = sm->lists.expert[j] * 2 * a.inter + (li - s_tiles - j * e_tiles) * 8;
        }
      }
    }
  };
  fill();          // of the shared expert
  wait_before();   // the choice
  let_next_begin();
  Lists& L = sm->lists;
  make_lists<true>(p, L);
  const int na = L.n_active;
  n_tiles = s_tiles + na * e_tiles;
  if (li >= s_tiles && li < n_tiles) {
    const int j = (li - s_tiles) / e_tiles;
    ly = L.expert[j] * 2 * a.inter + (li - s_tiles - j * e_tiles) * 8;
  }

  const int g = lane >> 2, t4 = lane & 3;
  int cs = 0, flip = 0;
  uint32_t ph = 0;
  for (int i = i0; i < n_tiles; i += tile_step) {
    const bool shared = i < s_tiles;
    const int j = shared ? -1 : (i - s_tiles) / e_tiles, r0 = (shared ? i : i - s_tiles - j * e_tiles) * 8;
    const int col0 = shared ? 0 : L.base[j], cnt = shared ? a.tokens : L.base[j + 1] - col0;
    const uint16_t* x[NG];       // the rows of this lane's columns
    float acc[NG][4];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      if (n > 0 && 8 * n >= cnt) continue;
      const int c = min(8 * n + g, cnt - 1);
      x[n] = a.x + (size_t)(shared ? c : (int)L.pair_t[col0 + c]) * a.hidden + t4 * 8;
    }
#pragma unroll
    for (int n = 0; n < NG; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
    // a chunk's activations, asked for one chunk ahead; lanes past the expert's tokens
    // ask for none (the requests of all 32 lanes take the load unit 64 clocks)
    uint4 b[4] = {};
    const auto load_x = [&](int k) {
      if (g >= cnt) return;
      if (k + kCols <= a.hidden) {
#pragma unroll
        for (int h = 0; h < 4; ++h) b[h] = *reinterpret_cast<const uint4*>(x[0] + k + 32 * h);
      } else {
        const int left = a.hidden - k - t4 * 8;                // columns from this lane's first on
#pragma unroll
        for (int h = 0; h < 4; ++h)
          b[h] = 32 * h < left ? *reinterpret_cast<const uint4*>(x[0] + k + 32 * h) : make_uint4(0, 0, 0, 0);
      }
    };
    load_x(member * kCols);
    for (int c = member; c < h_chunks; c += kTeam) {
      const int k = c * kCols, left = a.hidden - k - t4 * 8;
      fill();                    // the stage before's place, while these are on their way
      ok = ok && moe_wait(a, &full[cs], ph);
      Frag f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) load_a(f[h], ring + cs * kStage, h * 8 + g, kStage / 2, t4);
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        if (n > 0 && 8 * n >= cnt) break;
        // the next group's activations are asked for before this one's products while
        // there are registers, after them with eight groups
        uint4 bm[4] = {};
        const auto load_group = [&](uint4* to) {
          if (n + 1 < NG && 8 * (n + 1) < cnt) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              to[q] = 32 * q < left && 8 * (n + 1) + g < cnt
                          ? *reinterpret_cast<const uint4*>(x[n + 1 < NG ? n + 1 : 0] + k + 32 * q)
                          : make_uint4(0, 0, 0, 0);
          }
        };
        if (NG <= 4) load_group(bm);
        // short chains of products, summed by the fp32 units: the tensor cores cut off
        // what an addition drops (one chain per row and the fast exponential in silu:
        // 1e-6 of the fp32 result; so: 2.6e-7, where plain fp32 products have 3.3e-7)
        float d[2][4] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (k + 64 * h < a.hidden) mma_block(d[h], f[h], b + 2 * h);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[n][q] += d[0][q] + d[1][q];
        if (NG <= 4) {
#pragma unroll
          for (int q = 0; q < 4; ++q) b[q] = bm[q];
        } else {
          load_group(b);
        }
      }
      load_x(k + kTeam * kCols);
      __syncwarp();
      ++free_stages;
      if (++cs == kStages) {
        cs = 0;
        ph ^= 1u;
      }
    }
    fill();
    // the team's four sums, in their order; lane (g, t4) of the first warp holds gate and
    // up of row g for columns 2 t4 and 2 t4 + 1
    const int cols = shared ? a.shared_inter : a.inter;
    uint16_t* const act = shared ? p.s_act : p.act;
    const size_t plane = (size_t)(shared ? a.tokens : a.tokens * a.top_k) * cols;
#pragma unroll
    for (int n = 0; n < NG; ++n)
      if (8 * n < cnt) {
        if (member > 0) sm->red[flip][warp][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * kTeam) : "memory");
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
              const float v = acc[n][o] / (1.0f + expf(-acc[n][o])) * acc[n][2 + o] * (shared ? __ldcg(&p.choice->shared_w[c]) : L.pair_w[col0 + c]);
              uint16_t hi = f32_to_bf16(v);
              if ((hi & 0x7fff) == 0x7f80 && isfinite(v)) --hi;   // the largest bf16
              const size_t at = (size_t)(col0 + c) * cols + r0 + g;
              const float rest = isinf(v) ? 0.0f : v - bf16_to_f32(hi);   // exact
              const uint16_t lo = f32_to_bf16(rest);
              act[at] = hi;
              act[plane + at] = lo;
              if (a.out_f32) act[2 * plane + at] = f32_to_bf16(rest - bf16_to_f32(lo));
            }
          }
        }
        flip ^= 1;
      }
  }
}

template <int P>   // parts of an activation
__global__ void __launch_bounds__(kMoeThreads, 1)
    moe_down_kernel(const __grid_constant__ MoeMaps maps, const __grid_constant__ MoeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const MoeArgs& a = p.a;
  const uint32_t raw = tc::smem_u32(smem), pad = (1024u - (raw & 1023u)) & 1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x, grid = gridDim.x;
  ProductSmem* sm = reinterpret_cast<ProductSmem*>(smem + pad + kRing);
  uint8_t* const ring = smem + pad + warp * kStages * kStage;          // this warp's
  const uint32_t ring_a = raw + pad + warp * kStages * kStage;
  uint64_t* const full = sm->full[warp];
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) tc::mbar_init(&full[s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // The choice was complete before the launch that ran the gate and up products let
  // this one begin; only its activations are still to come.
  Lists& L = sm->lists;
  make_lists<false>(p, L);
  const int i_chunks = (a.inter + kCols - 1) / kCols, s_chunks = (a.shared_inter + kCols - 1) / kCols;

  // A team takes every fourth expert, its four warps every fourth chunk; of the shared
  // expert a warp takes every sixteenth chunk.  A CTA begins with its own one of the
  // experts, so that the CTAs do not all read the same activations at once.  All
  // this hangs on the experts', the chunks' and the CTA's numbers alone.
  const int team = warp / kTeam, member = warp % kTeam, n_team = L.n_team[team];
  const uint32_t* const of_team = L.of_team[team];
  int start = 0;
  {
    const int from = (int)((long long)cta * a.experts / grid);
    for (int lo = 0, hi = n_team; lo < hi;) {   // the first one not below `from`
      const int mid = (lo + hi) >> 1;
      if (Entry::expert(of_team[mid]) < from) lo = mid + 1; else hi = mid;
      start = lo;
    }
    if (start == n_team) start = 0;
  }
  // This warp's chunks in order, the loads kStages ahead of the products: of output
  // tile i, expert j (the team's n-th; at n = -1 the shared one), chunk c.
  const uint32_t all = Entry::kShared | Entry::of(0, 0, a.tokens);
  struct Walk {
    int i, n;
    uint32_t j;
    int c;
  };
  const auto settle = [&](Walk& w) {     // on to the first chunk from w on that exists
    while (w.c >= (Entry::shared(w.j) ? s_chunks : i_chunks)) {
      if (++w.n >= n_team) {
        w.n = -1;
        w.i += grid;
        if (w.i >= p.tiles3) return;
        w.j = all;
        w.c = warp;
      } else {
        w.j = of_team[start + w.n < n_team ? start + w.n : start + w.n - n_team];
        w.c = member;
      }
    }
  };
  Walk l{cta, -1, all, warp};
  if (l.i < p.tiles3) settle(l);
  // loaded and not yet multiplied, oldest first
  constexpr int kEnd = 0x7fffffff;
  int qi[kStages], qc[kStages], ls = 0, queued = 0;
  uint32_t qj[kStages];
#pragma unroll
  for (int s = 0; s < kStages; ++s) qi[s] = kEnd;
  bool ok = true;   // after a wait that gave up no later one waits, and nothing more is asked for
  const auto fill = [&]() {
    while (ok && queued < kStages && l.i < p.tiles3) {
      const bool shared = Entry::shared(l.j);
      if (lane == 0)
        load_stage<false>(ring_a + ls * kStage, &full[ls], shared ? &maps.s_whole : &maps.whole,
                   shared ? &maps.s_edge : &maps.edge, shared ? a.shared_inter : a.inter, l.c, p.rows3,
                   Entry::expert(l.j) * a.hidden + l.i * p.rows3, -1);
      __syncwarp();
#pragma unroll
      for (int s = 0; s < kStages; ++s)
        if (s == queued) {
          qi[s] = l.i;
          qj[s] = l.j;
          qc[s] = l.c;
        }
      ++queued;
      if (++ls == kStages) ls = 0;
      l.c += shared ? kMoeWarps : kTeam;
      settle(l);
    }
  };
  fill();
  // The activations.  (The next call's router is not let begin before this kernel ends:
  // its CTAs then gathered on the SMs that were free first, 126 us for 118 at 16 tokens.)
  wait_before();

  const int g = lane >> 2, t4 = lane & 3;
  int cs = 0;
  uint32_t ph = 0;
  // Columns 8 n .. of an expert (pairs base + 8 n ..): this lane's activations.
  const int np = a.tokens * a.top_k;
  const auto load_act = [&](uint4 (&x)[P][4], uint32_t j, int c, int n) {
    const bool shared = Entry::shared(j);
    const int cols = shared ? a.shared_inter : a.inter;
    const int k = c * kCols + t4 * 8, base = Entry::base(j), cnt = Entry::count(j);
    // (lanes past the last pair ask for nothing: most experts have one token, and the
    // requests of all 32 lanes, 7 of 8 for zeros, took the load unit 64 clocks a
    // warp: 204 us for 64 tokens where 135 now are.  What they hold meets only
    // columns that nobody reads.)
    if (8 * n + g >= cnt) return;
    const uint16_t* row = (shared ? p.s_act : p.act) + ((size_t)(base + 8 * n + g) * cols + k);
    const size_t plane = (size_t)(shared ? a.tokens : np) * cols;
    if ((c + 1) * kCols <= cols) {
#pragma unroll
      for (int part = 0; part < P; ++part)
#pragma unroll
        for (int h = 0; h < 4; ++h) x[part][h] = __ldcg(reinterpret_cast<const uint4*>(row + part * plane + 32 * h));
    } else {
#pragma unroll
      for (int part = 0; part < P; ++part)
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          x[part][h] = make_uint4(0, 0, 0, 0);
          if (k + 32 * h < cols) x[part][h] = __ldcg(reinterpret_cast<const uint4*>(row + part * plane + 32 * h));
        }
    }
  };
  float* const sums = reinterpret_cast<float*>(sm->red);
  float* const mine = sums + warp * a.tokens * kSumRow;
  uint4 x[P][4] = {};            // of the first 8 columns, asked for one chunk ahead
  if (qi[0] != kEnd) load_act(x, qj[0], qc[0], 0);
  for (int i = cta; i < p.tiles3; i += grid) {
    for (int k = lane; k < a.tokens * kSumRow; k += 32) mine[k] = 0.0f;
    __syncwarp();
    while (qi[0] == i) {
      const uint32_t j = qj[0];
      const int c = qc[0];
      const bool shared = Entry::shared(j);
      const int cols = shared ? a.shared_inter : a.inter, base = Entry::base(j), cnt = Entry::count(j);
      // where this lane's first two columns add up
      int to[2];
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int col = 2 * t4 + o;
        to[o] = shared ? col : (col < cnt ? (int)L.pair_t[base + col] : 0);
      }
      ok = ok && moe_wait(a, &full[cs], ph);
      Frag f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) load_a(f[h], ring + cs * kStage, h * p.rows3 + g, 1024, t4);
      for (int n = 0; 8 * n < cnt; ++n) {
        if (n > 0) {
          load_act(x, j, c, n);
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const int col = 8 * n + 2 * t4 + o;
            to[o] = shared ? col : (col < cnt ? (int)L.pair_t[base + col] : 0);
          }
        }
        // four chains: a product's latency is 38 clocks
        float acc[2][4] = {}, low[2][4] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (c * kCols + 64 * h < cols) {
            mma_block(acc[h], f[h], x[0] + 2 * h);
#pragma unroll
            for (int part = 1; part < P; ++part) mma_block(low[h], f[h], x[part] + 2 * h);
          }
        // lane (g, t4) holds rows g, g + 8 of columns 2 t4, 2 t4 + 1
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const int col = 8 * n + 2 * t4 + o;
          if (col < cnt) {
            float* y = mine + to[o] * kSumRow + g;
            y[0] += (acc[0][o] + acc[1][o]) + (low[0][o] + low[1][o]);
            y[8] += (acc[0][2 + o] + acc[1][2 + o]) + (low[0][2 + o] + low[1][2 + o]);
          }
        }
      }
      __syncwarp();
      if (++cs == kStages) {
        cs = 0;
        ph ^= 1u;
      }
#pragma unroll
      for (int s = 0; s + 1 < kStages; ++s) {
        qi[s] = qi[s + 1];
        qj[s] = qj[s + 1];
        qc[s] = qc[s + 1];
      }
      qi[kStages - 1] = kEnd;
      --queued;
      if (qi[0] != kEnd) load_act(x, qj[0], qc[0], 0);
      fill();                    // while the activations are on their way
    }
    __syncthreads();
    for (int k = tid; k < a.tokens * 16; k += kMoeThreads) {
      const int r = k & 15, t = k >> 4, h = i * p.rows3 + r;
      if (r < p.rows3 && h < a.hidden) {
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < kMoeWarps; ++q) v += sums[(q * a.tokens + t) * kSumRow + r];
        const size_t at = (size_t)t * a.hidden + h;
        if (a.out_f32)
          static_cast<float*>(a.y)[at] = v;
        else
          static_cast<uint16_t*>(a.y)[at] = f32_to_bf16(v);
      }
    }
    __syncthreads();
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

// A launch that may begin while the one before it in the stream still runs.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, uint32_t smem, cudaStream_t stream,
                         Args... args) {
  cudaError_t e;
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
    return e;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int NG>
cudaError_t launch_products(const MoeMaps& up, const MoeMaps& down, const MoeParams& p, int sms, cudaStream_t stream) {
  cudaError_t e = launch_early(moe_gate_up_kernel<NG>, dim3(sms), kMoeThreads, kGateUpSmem, stream, up, p);
  if (e != cudaSuccess) return e;
  return launch_early(p.a.out_f32 ? moe_down_kernel<3> : moe_down_kernel<2>, dim3(p.tiles3 < sms ? p.tiles3 : sms),
                      kMoeThreads, down_smem(p.a.tokens), stream, down, p);
}

}  // namespace

size_t moe_scratch_bytes(int tokens, int, int inter, int experts, int top_k, int shared_inter) {
  const size_t T = tokens > 0 ? tokens : 1;
  return up256(sizeof(Choice)) + up256(T * (experts + 1) * 8) + up256(T * top_k * inter * 6) +
         up256(T * shared_inter * 6);
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
  p.choice = reinterpret_cast<Choice*>(ws);
  ws += up256(sizeof(Choice));
  p.logit = reinterpret_cast<float2*>(ws);
  ws += up256(T * (a.experts + 1) * 8);
  p.act = reinterpret_cast<uint16_t*>(ws);
  ws += up256(T * a.top_k * a.inter * 6);
  p.s_act = reinterpret_cast<uint16_t*>(ws);
  // output rows: tiles of at most 16, as many as give every CTA the same number
  const int per = (a.hidden + 16 * sms - 1) / (16 * sms);
  p.rows3 = (a.hidden + per * sms - 1) / (per * sms);
  p.tiles3 = (a.hidden + p.rows3 - 1) / p.rows3;
  MoeMaps up, down;
  if (!weight_maps(&up.whole, &up.edge, a.w_gate_up, (uint64_t)a.experts * 2 * a.inter, a.hidden, 8) ||
      !weight_maps(&down.whole, &down.edge, a.w_down, (uint64_t)a.experts * a.hidden, a.inter, p.rows3))
    return cudaErrorInvalidValue;
  if (a.shared_inter > 0 &&
      (!weight_maps(&up.s_whole, &up.s_edge, a.s_gate_up, 2ull * a.shared_inter, a.hidden, 8) ||
       !weight_maps(&down.s_whole, &down.s_edge, a.s_down, a.hidden, a.shared_inter, p.rows3)))
    return cudaErrorInvalidValue;
  const int rows = a.experts + (p.a.s_gate ? 1 : 0);
  const int nt = a.tokens == 1 ? 1 : 8;   // eight tokens share an expert's row
  const auto router = nt == 1 ? moe_router_kernel<1> : moe_router_kernel<8>;
  if ((e = launch_early(router, dim3((rows + 7) / 8, (a.tokens + nt - 1) / nt), 32 * kRouterWarps, kRouterSmem, stream,
                        p)) != cudaSuccess)
    return e;
  if ((e = launch_early(moe_choice_kernel, dim3(a.tokens), kChoiceThreads, 0, stream, p)) != cudaSuccess) return e;
  if (a.tokens <= 8) return launch_products<1>(up, down, p, sms, stream);
  if (a.tokens <= 16) return launch_products<2>(up, down, p, sms, stream);
  if (a.tokens <= 32) return launch_products<4>(up, down, p, sms, stream);
  return launch_products<8>(up, down, p, sms, stream);
}

}  // namespace gdn
