// gdn_attn_shared.cu -- attention of a batch of sequences that share a long
// prefix, each with a paged tail of its own (tcgen05 tensor cores).
//
// Mathematics.  Row r = (sequence, step, query head) wants
//   o = sum_j e^{s_j - m} v_j / sum_j e^{s_j - m},  s_j = scale q.k_j,
// over the prefix's keys and then its tail's.  Any partition of the keys into
// ranges can be summed apart: a range leaves (m, l = sum e^{s - m}, O = sum
// e^{s - m} v), and ranges join as sum 2^{m_i - M} O_i / sum 2^{m_i - M} l_i.
//
// Jobs.  The rows of one key head meet the prefix together: 256 rows (whole
// tokens of h_q / h_kv heads) by the prefix's keys is one job, a dense product
// that reads the prefix once per 256 rows instead of once per row.  A
// sequence's tail by its own steps * h_q / h_kv rows is another, bound by its
// bytes.  Both are rows x keys x d products and run through the same pipeline;
// a tail's unused rows of the 256 cost tensor time that its loads hide.
//
// Split.  All jobs' tiles of 128 keys are laid end to end, weighted by what a
// tile costs, and every pair of CTAs (one per SM) takes an equal share, so a single
// long prefix fills the GPU as well as many short tails do.  A share ends
// where it ends, inside a job if need be: a job's ranges are joined by a
// second launch.  The shares follow from the lengths alone, so equal calls add
// in equal order.  Each pair sums the tails' costs itself from tail_len on the
// device; the host needs no lengths, and a captured step stays valid.
//
// Pair.  The two CTAs of a cluster hold 128 rows each and run one product
// (cta_group::2): each brings half of the keys of K and half of the dimensions
// of V, so a tile costs an SM half the shared memory and half the L2 traffic it
// would cost alone.  (With one CTA per job of 128 rows at d = 256, the five
// stages that fit beside q held 1.25 tiles, and a tile took 4600 clocks for
// 2048 of products.)
//
// Pipeline per pair, over its tiles without a pause between jobs:
//   warp 0     TMA, each CTA its half: q tiles, K and V in a ring of stages, all
//              reported to the first CTA
//   warp 1     of the first CTA, for both: S = Q K^T
//   warp 10    likewise: O += P V.  (One warp for both products left the tensor
//              cores idle for some 500 clocks at each change between them, 1000
//              of a tile's 3400; now one's barriers pass under the other's
//              products.)
//   warp 11    a tail's last V tile: zeros in the rows past its end, and for infinities
//              and NaN of tokens that not all of its queries see
//   warps 2-9  softmax: a thread holds half a row's 128 scores; P goes back to
//              tensor memory as bf16 and is read from there as the A operand
// TMEM: O (d columns), one score tile (128), two weight tiles (64 each).  The
// scores' place is free again as soon as they are in registers, so the next
// tile's scores are computed under this one's exponentials and O product (with
// two score tiles and the weights written over them, each score product waited
// for the O product two tiles back: 2880 clocks a tile).  O is rescaled only
// when a row's maximum has grown by more than 8 binary orders (P <= 2^8 fits
// bf16 as well as P <= 1 does, and the sums are fp32), so almost never.
//
// Measured, both launches: 64 sequences on a prefix of 32768 (16 query heads, 2 key
// heads, d = 256) 50 us, 690 TFLOP/s of useful products; 256 sequences on 32768
// 168 us, 830; 256 on 4096 with tails up to 3000 169 us, 4.9 TB/s; one sequence
// of 833 keys 13 us, all latency.  A prefix tile takes some 2700 clocks: 2048 of
// products, next to 2000 of softmax on the other side of the same barriers; a
// tail's tile costs as many clocks of products for its few rows.  The rest of a call
// is 2.5 us before the first tile and 8 to 10 in the join.  Tables of 16-row pages
// cost 16 copies a tile instead of 4, some 150 clocks each: pages of 64 rows or
// more are better (17 sequences of 4 steps on 5000, pages of 16: 43 us, of which 1.3
// for the look at the tails' last values).
//
// Masks.  A masked key's weight is zero, but zero times an infinity is NaN, and one
// product serves all rows of a job.  So what the product reads of V is finite
// wherever some row does not see it: rows past a job's end are zeros, and of a
// tail's last steps - 1 tokens, which its earlier queries do not see, infinities
// and NaN are.  The join adds those to the rows that do see them (a positive weight
// times an infinity is that infinity).
//
// Rounding: weights P to bf16 (half a step, 2^-8 of each weight), because the
// tensor cores take both operands in one 16-bit type; scores, maxima, sums and
// outputs stay fp32 until the one rounding of the result.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "../../include/gdn.h"
#include "gdn_attn_ranges.h"
#include "gdn_common.cuh"
#include "gdn_launch.h"
#include "gdn_prefill.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kTile = 128;            // keys per tile
constexpr int kMaxShares = 80;        // CTA pairs the workspace has room for
constexpr int kThreads = 384;
constexpr int kSoftWarps = 8;
constexpr int kPvWarp = 2 + kSoftWarps, kCleanWarp = kPvWarp + 1;
constexpr int kMaxStages = 8;
constexpr uint32_t kCtrlBytes = 3 * 1024;

// What a tile costs, in quarters of a prefix tile, and a job's fixed part (its rows
// in and out).  A tail's tile by itself takes a fifth longer, for its loads, but then
// the memory is what all pairs share: at 256 sequences of 4096 + tails a weight of
// 4.5 took 177 us for 167, at 64 of 32768 55 for 52.
constexpr int kCostPrefix = 4, kCostTail = 4, kCostJob = 2;

// Shape of one call, the same for both launches.
struct Plan {
  int ntok, h_kv, G, R;        // query tokens, key heads, group, rows of a tail job
  int tpb, nmb;                // tokens per CTA of a prefix job, prefix jobs per key head
  int np, shares;              // prefix jobs, shares (CTA pairs)
  long long ptiles;            // prefix tiles
  long long wp;                // cost of all prefix jobs
};

struct SharedParams {
  AttnSharedArgs a;
  Plan pl;
  int2* span;                  // per job: the first and the last share with a range of it
  uint8_t* hidden;             // per tail job [last tile with hidden tokens, the one before][CTA]: any not finite
  float4* ml;                  // (m, l half 0, l half 1, -) per slot row
  float* opart;                // per slot: [d / 4][rows][4]
};

template <int D>
struct Cfg {
  static constexpr uint32_t STAGE = 128 * D;            // 64 keys of K, or 128 keys of half of V's dimensions
  static constexpr int NK = D == 256 ? 3 : (D == 128 ? 6 : 8), NV = D == 256 ? 2 : NK;   // stages
  static constexpr uint32_t QBYTES = 128 * D * 2;
  static constexpr uint32_t SMEM = kCtrlBytes + QBYTES + (NK + NV) * STAGE;
  static constexpr uint32_t IDESC_QK = tc::idesc_bf16(256, kTile, 0, 0);
  static constexpr uint32_t IDESC_PV = tc::idesc_bf16(256, D, 0, 1);
  static constexpr uint64_t DESC_K = tc::sdesc_sw128(16, 1024);
  // V: rows of VROW bytes, half of the dimensions in blocks of up to 64; at d = 64
  // a half is 32 dimensions and the swizzle spans 64 bytes
  static constexpr int VROW = D == 64 ? 64 : 128, VBLK = D == 64 ? 1 : D / 128;
  static constexpr uint32_t T_S = 256, T_P = 384;       // TMEM columns of the scores, the weights
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(NK <= kMaxStages && NV <= kMaxStages && NK >= 2, "barriers");
};

// Descriptor of V read MN-major; blocks of dimensions are `lbo` bytes apart.
template <int D>
__device__ __forceinline__ uint64_t desc_v(uint32_t lbo) {
  const uint64_t sw = D == 64 ? 4 : 2;   // 64- or 128-byte swizzle
  return (static_cast<uint64_t>((lbo >> 4) & 0x3FFF) << 16) |
         (static_cast<uint64_t>((8 * Cfg<D>::VROW) >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (sw << 61);
}

struct Ctrl {
  uint64_t k_full[kMaxStages], v_full[kMaxStages];
  uint64_t s_full[kMaxStages];    // a tile's scores are done, and so is its K stage
  uint64_t pv_done[kMaxStages];   // a tile's O product is done, and so is its V stage
  uint64_t q_full[2], q_done[2], p_ready[2];
  uint64_t s_free;                // the scores are in registers
  uint64_t landed[kMaxStages];    // this CTA's half of a V tile that is to be cleaned, by its stage
  uint64_t seg_done;              // a segment's last O product
  uint64_t pair[4];            // the two warps of a row quarter
  uint32_t tmem;
  int job0;
  long long x0, x1, pos0;
  float red[2][2][128];        // row maxima of a half tile, by tile parity
};
static_assert(sizeof(Ctrl) <= kCtrlBytes, "control block");

__device__ __forceinline__ void arrive(uint64_t* mbar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(mbar)) : "memory");
}
// Address of the pair's CTA `rank`'s copy of a shared variable.
__device__ __forceinline__ uint32_t peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Boxes into this CTA's shared memory, reported to `mbar` of either CTA of the pair.
__device__ __forceinline__ void tma_pair(void* dst, const CUtensorMap* tm, int x, int y, int z, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4}], [%5];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(mbar)
      : "memory");
}

// D[tmem] (+)= A B^T over the pair, one K = 16 step: A in shared memory, or in
// tensor memory (_ts).
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void mma_pair_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
// Both CTAs' copies of the mbarrier arrive once the products issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* mbar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          tc::smem_u32(mbar)),
      "h"((uint16_t)3)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a maximum is subtracted as: where no score but -inf (or NaN) was met, 0.
__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.0f : m; }

// Shares in use: none is shorter than a tile, so that the shares from a job's first
// range to its last all have one.
__device__ __forceinline__ int shares_of(const Plan& pl, long long total) {
  constexpr int top = kCostPrefix > kCostTail ? kCostPrefix : kCostTail;
  return (int)max(1LL, min((long long)pl.shares, total / top));
}
__device__ __forceinline__ int tail_tiles(int len) { return (len + kTile - 1) / kTile; }
__device__ __forceinline__ long long tail_cost_of(int len) {
  return len > 0 ? (long long)tail_tiles(len) * kCostTail + kCostJob : 0;
}
// Tiles of a job that starts at `pos` which lie before x.  What is divided is
// below n times a tile's cost, 2^24 * 4, so 32 bits hold it (64-bit divisions by a
// variable in this walk took 6 us of a call of 61).
__device__ __forceinline__ int tiles_before(long long x, long long pos, bool prefix, int n) {
  const long long q = x - pos - kCostJob;
  if (q <= 0) return 0;
  if (q >= (long long)n * (prefix ? kCostPrefix : kCostTail)) return n;
  return (int)(prefix ? (uint32_t)q / kCostPrefix : (uint32_t)q / kCostTail);
}
// A tail's length, clamped into its table.
__device__ __forceinline__ int clamp_tail(const AttnSharedArgs& a, int n) {
  const int top = a.tail_width * a.page;
  return n < 0 ? 0 : (n > top ? top : n);
}
__device__ __forceinline__ int tail_length(const AttnSharedArgs& a, int b) {
  return a.tail_width == 0 ? 0 : clamp_tail(a, a.tail_len[b]);
}

// Walks the tiles of one share, job by job.  Every role keeps its own.
struct Cursor {
  long long pos;       // cost position of the job `job`
  long long x0, x1;
  int job;             // next job to look at
  int len;             // of the current sequence's tail (jobs of one sequence are adjacent)
  int ahead;           // tail_len of the next sequence, on its way
  int seg;             // segments begun, minus one
  // the current segment
  bool prefix, valid, first, last;
  int hk, mb;          // key head; block of rows (prefix) or sequence (tail)
  int slot_job;        // prefix job, or tail job
  int t, t0, t1, keys; // tile, the range's first and end, keys of the job

  __device__ __forceinline__ void init(const SharedParams& p, const Ctrl* c) {
    pos = c->pos0;
    x0 = c->x0;
    x1 = c->x1;
    job = c->job0;
    len = ahead = -1;
    seg = -1;
    t = t0 = t1 = 0;
    valid = true;
    find(p);
  }
  __device__ __forceinline__ void find(const SharedParams& p) {
    const Plan& pl = p.pl;
    const int njobs = pl.np + p.a.batch * pl.h_kv;
    while (true) {
      if (job >= njobs || pos >= x1) {
        valid = false;
        return;
      }
      long long cost;
      int n;
      prefix = job < pl.np;
      if (prefix) {
        hk = job / pl.nmb;
        mb = job - hk * pl.nmb;
        slot_job = job;
        n = (int)pl.ptiles;
        keys = (int)p.a.prefix_len;
        cost = pl.ptiles * kCostPrefix + kCostJob;
      } else {
        slot_job = job - pl.np;
        mb = slot_job / pl.h_kv;
        hk = slot_job - mb * pl.h_kv;
        if (hk == 0 || len < 0) {
          len = len < 0 ? tail_length(p.a, mb) : clamp_tail(p.a, ahead);
          if (p.a.tail_width > 0 && mb + 1 < p.a.batch) ahead = p.a.tail_len[mb + 1];
        }
        n = tail_tiles(len);
        keys = len;
        cost = tail_cost_of(len);
      }
      const int a = tiles_before(x0, pos, prefix, n), b = tiles_before(x1, pos, prefix, n);
      pos += cost;
      ++job;
      if (a < b) {
        t = t0 = a;
        t1 = b;
        first = true;
        last = a + 1 == b;
        ++seg;
        return;
      }
    }
  }
  __device__ __forceinline__ void next(const SharedParams& p) {
    if (++t < t1) {
      first = false;
      last = t + 1 == t1;
    } else {
      find(p);
    }
  }
  // keys of the current tile
  __device__ __forceinline__ int count() const {
    return min(keys - t * kTile, kTile);
  }
};

// Whether a tile's V passes the cleaning warp before its product: a tail or a prefix
// ends in it inside 16 keys, or it holds some of the last steps - 1 tokens of a tail.
template <bool several>
__device__ __forceinline__ bool cleaned(const AttnSharedArgs& a, const Cursor& c) {
  return (c.count() & 15) != 0 || (several && !c.prefix && c.keys - c.t * kTile < kTile + a.steps - 1);
}

// Infinities and NaN of two bf16; zeros in a finite one's place.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u ? w & 0xffffu : 0u) | ((w & 0x7f800000u) == 0x7f800000u ? w & 0xffff0000u : 0u);
}

// Position in a ring of N stages.
template <int N>
struct Ring {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void step() {
    if (++s == N) {
      s = 0;
      ph ^= 1u;
    }
  }
};

// One wait of a role: false (and the status word) when it gave up.
__device__ __forceinline__ bool wait_for(const AttnSharedArgs& a, uint64_t* mbar, uint32_t parity) {
  // the usual case, without the clock
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred P1;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 P1, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, P1;\n\t}\n"
      : "=r"(done)
      : "r"(tc::smem_u32(mbar)), "r"(parity)
      : "memory");
  if (done || tc::mbar_wait(mbar, parity, kWaitBudget)) return true;
  record_status(a.status, GDN_ERR_DEVICE_TIMEOUT);
  return false;
}

// 64 scores of this thread's row: both loads in flight, one wait.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
  uint32_t r[64];
#define GDN_LD32(o, at)                                                                                          \
  asm volatile(                                                                                                  \
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%"  \
      "18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"                                          \
      : "=r"(r[o + 0]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]),          \
        "=r"(r[o + 6]), "=r"(r[o + 7]), "=r"(r[o + 8]), "=r"(r[o + 9]), "=r"(r[o + 10]), "=r"(r[o + 11]),        \
        "=r"(r[o + 12]), "=r"(r[o + 13]), "=r"(r[o + 14]), "=r"(r[o + 15]), "=r"(r[o + 16]), "=r"(r[o + 17]),    \
        "=r"(r[o + 18]), "=r"(r[o + 19]), "=r"(r[o + 20]), "=r"(r[o + 21]), "=r"(r[o + 22]), "=r"(r[o + 23]),    \
        "=r"(r[o + 24]), "=r"(r[o + 25]), "=r"(r[o + 26]), "=r"(r[o + 27]), "=r"(r[o + 28]), "=r"(r[o + 29]),    \
        "=r"(r[o + 30]), "=r"(r[o + 31])                                                                         \
      : "r"(at))
  GDN_LD32(0, taddr);
  GDN_LD32(32, taddr + 32);
#undef GDN_LD32
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

// 16-byte piece `c16` of a row of a V stage, whose pieces of pages are `rpb` rows.
template <int D>
__device__ __forceinline__ uint4* v_chunk(uint8_t* v, int row, int c16, int rpb) {
  constexpr int VROW = Cfg<D>::VROW, per = VROW / 16;
  const int in = row & (rpb - 1);
  return reinterpret_cast<uint4*>(v + (row - in) * D + (c16 / per) * (rpb * VROW) + in * VROW + (c16 % per) * 16);
}

// Zeros for the infinities and NaN in rows [from, n) of a V stage, by one warp;
// whether there were any.  (Not inlined, and not in the kernel for one query token:
// in that kernel's body it cost the prefix's tiles, which never come here, 1000 clocks
// each, 49 -> 56 us for 64 sequences, and as a call still 1 us.)
template <int D>
__device__ __noinline__ bool clear_not_finite(uint8_t* v, int from, int n, int rpb) {
  bool found = false;
  for (int w = threadIdx.x & 31; w < (n - from) * (D / 16); w += 32) {
    uint4* const at = v_chunk<D>(v, from + w / (D / 16), w % (D / 16), rpb);
    const uint4 x = *at;
    const uint4 bad = make_uint4(not_finite(x.x), not_finite(x.y), not_finite(x.z), not_finite(x.w));
    if (bad.x | bad.y | bad.z | bad.w) {
      *at = make_uint4(x.x ^ bad.x, x.y ^ bad.y, x.z ^ bad.z, x.w ^ bad.w);
      found = true;
    }
  }
  return __any_sync(0xffffffffu, found);
}

// several: more than one query token a sequence.
template <int D, bool several>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    attn_shared_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_qp, const __grid_constant__ CUtensorMap tm_qt,
                       const __grid_constant__ SharedParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctrl* ctl = reinterpret_cast<Ctrl*>(smem);
  const AttnSharedArgs& a = p.a;
  const Plan& pl = p.pl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = tc::smem_u32(smem);
  uint8_t* const qs = smem + kCtrlBytes;
  uint8_t* const ring = qs + C::QBYTES;           // K stages, then V stages
  const uint32_t rank = blockIdx.x & 1u;
  const int share = blockIdx.x >> 1;
  if (base & 1023u) {   // the swizzle atoms need it; shared memory starts there (in both CTAs alike)
    record_status(a.status, GDN_ERR_CUDA);
    return;
  }

  if (warp == kCleanWarp) {
    if (lane < kMaxStages) {
      tc::mbar_init(&ctl->k_full[lane], 1);
      tc::mbar_init(&ctl->v_full[lane], 2);
      tc::mbar_init(&ctl->landed[lane], 1);
      tc::mbar_init(&ctl->s_full[lane], 1);
      tc::mbar_init(&ctl->pv_done[lane], 1);
    } else if (lane < kMaxStages + 2) {
      tc::mbar_init(&ctl->q_full[lane - kMaxStages], 1);
      tc::mbar_init(&ctl->q_done[lane - kMaxStages], 1);
      tc::mbar_init(&ctl->p_ready[lane - kMaxStages], 2 * kSoftWarps);
    } else if (lane < kMaxStages + 6) {
      tc::mbar_init(&ctl->pair[lane - kMaxStages - 2], 2);
    } else if (lane == kMaxStages + 6) {
      tc::mbar_init(&ctl->s_free, 2 * kSoftWarps);
      tc::mbar_init(&ctl->seg_done, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // launched while the kernel before it runs: its results are there from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // Tensor memory only now: held before, it could be what the kernel before this one
  // waits for, and neither would end.
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::smem_u32(&ctl->tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  // ---- this pair's share: the running cost of the tails, then a search ----
  long long* scan = reinterpret_cast<long long*>(ring);   // [batch + 1] and warp totals, before the ring is used
  long long* wsum = scan + GDN_ATTN_MAX_BATCH + 8;
  long long tails = 0;
  if (a.tail_width > 0) {
    constexpr int PER = 4;
    static_assert(kThreads * PER >= GDN_ATTN_MAX_BATCH, "one pass");
    long long v[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = i * kThreads + threadIdx.x;
      v[i] = 0;
      if (b < a.batch) {
        const int n = a.tail_len[b];
        if ((n < 0 || n > a.tail_width * a.page) && blockIdx.x == 0) record_status(a.status, GDN_ERR_DEVICE_BOUNDS);
        v[i] = tail_cost_of(clamp_tail(a, n)) * pl.h_kv;
      }
    }
    // chunks of kThreads sequences, one after the other
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (i * kThreads >= a.batch) break;
      long long inc = v[i];
      for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, m);
        if (lane >= m) inc += o;
      }
      if (lane == 31) wsum[warp] = inc;
      __syncthreads();
      long long before = tails;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += wsum[w];
        sum += wsum[w];
      }
      const int b = i * kThreads + threadIdx.x;
      if (b < a.batch) scan[b] = before + inc - v[i];
      tails = sum;
      __syncthreads();
    }
  }
  if (threadIdx.x == 0) {
    const long long total = pl.wp + tails;
    const int shares = shares_of(pl, total);
    const long long x0 = share < shares ? total * share / shares : total;
    const long long x1 = share < shares ? total * (share + 1) / shares : total;
    ctl->x0 = x0;
    ctl->x1 = x1;
    if (x0 < pl.wp) {
      const long long cost = pl.ptiles * kCostPrefix + kCostJob;
      const long long j = x0 / cost;
      ctl->job0 = (int)j;
      ctl->pos0 = j * cost;
    } else if (x0 < total) {
      const long long x = x0 - pl.wp;
      int lo = 0, hi = a.batch;      // the last b with scan[b] <= x
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (scan[mid] <= x) lo = mid; else hi = mid;
      }
      ctl->job0 = pl.np + lo * pl.h_kv;
      ctl->pos0 = pl.wp + scan[lo];
    } else {                         // nothing to do
      ctl->job0 = pl.np + a.batch * pl.h_kv;
      ctl->pos0 = total;
    }
  }
  tc::fence_proxy_async();   // the scan's writes before the ring's copies
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();            // the other CTA's barriers are set up
  tc::fence_after_sync();
  const uint32_t tmem = ctl->tmem;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the q region holds two tail jobs' rows when they are few, else one
  const bool halves = pl.R <= 64;

  if (warp == 0) {
    // ---- loads ----
    // A page table entry is a trip to L2: lane j reads the entry of piece j of the
    // tile after next while this one's loads are issued (K and then V of a tile
    // use the same pieces).
    Cursor cn, ck, cv;
    cn.init(p, ctl);
    ck = cn;
    cv = cn;
    Ring<C::NK> rk;
    Ring<C::NV> rv;
    const int rpb = a.page < 64 ? a.page : 64;           // rows per box
    const int rsh = 31 - __clz(rpb), shift = 31 - __clz(a.page);
    bool ok = true, prev_whole = true;
    uint32_t loaded = 0, segs = 0;
    // the page where piece `lane` of c's tile lies, as the table has it: looked at only
    // when the tile is loaded, so that nothing waits for the table
    auto page_of = [&](const Cursor& c) -> int {
      if (!c.valid || (lane << rsh) >= c.count()) return 0;
      const int32_t* table = c.prefix ? a.prefix_pages : a.tail_pages + (size_t)c.mb * a.tail_width;
      return __ldg(table + ((c.t * kTile + (lane << rsh)) >> shift));
    };
    // the row of the cache where that piece begins
    auto row_of = [&](const Cursor& c, int pg) -> int {
      if (pg < 0 || pg >= a.n_pages) {
        record_status(a.status, GDN_ERR_DEVICE_BOUNDS);
        pg = 0;
      }
      return (int)(((long long)pg << shift) + ((c.t * kTile + (lane << rsh)) & (a.page - 1)));
    };
    int page_n = page_of(cn), rows_k = 0, rows_v = 0;
    const auto tile_rows = [&](int n) { return ((n + rpb - 1) >> rsh) << rsh; };   // rows of its boxes
    auto load_k = [&]() {
      if (ck.first) {
        const int s = ck.seg, h = s & 1;
        const bool whole = ck.prefix || !halves;
        if (s >= 2) ok = wait_for(a, &ctl->q_done[h], (uint32_t)((s >> 1) - 1) & 1u);
        if (ok && s >= 1 && (whole || prev_whole))
          ok = wait_for(a, &ctl->q_done[h ^ 1], (uint32_t)((s - 1) >> 1) & 1u);
        if (!ok) return;
        prev_whole = whole;
        ++segs;
        // a prefix job has rows in both CTAs, a tail in the first
        const uint32_t bytes = (uint32_t)(ck.prefix ? 2 * pl.tpb * pl.G : pl.R) * D * 2;
        const uint32_t mbar = peer(tc::smem_u32(&ctl->q_full[h]), 0);
        if (rank == 0 && lane == 0) mbar_expect_tx(&ctl->q_full[h], bytes);
        __syncwarp();
        if (lane < D / 64 && (ck.prefix || rank == 0))
          tma_pair(qs + lane * 16384 + (whole ? 0 : h * 8192), ck.prefix ? &tm_qp : &tm_qt, lane * 64, ck.hk * pl.G,
                   ck.prefix ? (2 * ck.mb + (int)rank) * pl.tpb : ck.mb * a.steps, mbar);
        __syncwarp();
      }
      const int n = ck.count();
      ok = wait_for(a, &ctl->s_full[rk.s], rk.ph ^ 1u);
      if (!ok) return;
      // both CTAs' boxes report to the first, which expects the bytes of all
      const uint32_t mbar = peer(tc::smem_u32(&ctl->k_full[rk.s]), 0);
      if (rank == 0 && lane == 0) mbar_expect_tx(&ctl->k_full[rk.s], (uint32_t)tile_rows(n) * (D * 2));
      __syncwarp();
      // this CTA's 64 keys: [block of 64 dimensions][64 keys][128 bytes]; pieces of
      // 64 keys come with all their blocks in one box
      const int mine = min(max(n - 64 * (int)rank, 0), 64), nb = (mine + rpb - 1) >> rsh;
      const int per = rpb == 64 ? 1 : D / 64;      // boxes per piece
      const int j = lane / per, d = lane - j * per;
      const int row = __shfl_sync(0xffffffffu, rows_k, (((int)rank * 64 >> rsh) + j) & 31);
      if (lane < nb * per)
        tma_pair(ring + rk.s * C::STAGE + d * 8192 + ((j * 128) << rsh), &tm_k, 0, row, ck.hk * (D / 64) + d, mbar);
      __syncwarp();
      rk.step();
    };
    auto load_v = [&]() {
      const int n = cv.count();
      ok = wait_for(a, &ctl->pv_done[rv.s], rv.ph ^ 1u);
      if (!ok) return;
      // as for K, with an arrival of each CTA; a tile to be cleaned reports to its own
      // CTA, whose cleaning warp then arrives
      uint32_t mbar = peer(tc::smem_u32(&ctl->v_full[rv.s]), 0);
      if (cleaned<several>(a, cv)) {
        mbar = peer(tc::smem_u32(&ctl->landed[rv.s]), rank);
        if (lane == 0) mbar_expect_tx(&ctl->landed[rv.s], (uint32_t)tile_rows(n) * D);
      } else if (lane == 0) {
        if (rank == 0) mbar_expect_tx(&ctl->v_full[rv.s], (uint32_t)tile_rows(n) * (D * 2));
        else arrive_at(mbar);
      }
      __syncwarp();
      // all keys of half of the dimensions: [piece][block of dimensions][keys][VROW bytes]
      const int nb = (n + rpb - 1) >> rsh;
      if (lane < nb)
        tma_pair(ring + (C::NK + rv.s) * C::STAGE + ((lane * D) << rsh), &tm_v, D == 64 ? 32 * (int)rank : 0, rows_v,
                 D == 64 ? cv.hk : cv.hk * (D / 64) + (int)rank * C::VBLK, mbar);
      __syncwarp();
      ++loaded;
      rv.step();
    };
    // ck steps to the tile cn has looked up, cn to the one after
    auto advance = [&]() {
      rows_v = rows_k;
      rows_k = row_of(cn, page_n);
      ck = cn;
      cn.next(p);
      page_n = page_of(cn);
    };
    if (ck.valid) {
      rows_k = row_of(cn, page_n);
      cn.next(p);
      page_n = page_of(cn);
      load_k();
      while (ok && cv.valid) {
        advance();
        if (ck.valid) load_k();
        if (!ok) break;
        load_v();
        cv = ck;
      }
      // the products' last reports have landed before the CTA ends
      for (uint32_t i = 1; i <= (uint32_t)C::NV && i <= loaded && ok; ++i)
        ok = wait_for(a, &ctl->pv_done[(loaded - i) % C::NV], ((loaded - i) / C::NV) & 1u);
      if (ok) ok = wait_for(a, &ctl->q_done[(segs - 1) & 1u], ((segs - 1) >> 1) & 1u);
    }
  } else if (warp == 1) {
    // ---- scores, by the first CTA for both ----
    Cursor c;
    c.init(p, ctl);
    Ring<C::NK> rk;
    bool ok = rank == 0;
    const uint32_t qa = base + kCtrlBytes, ra = qa + C::QBYTES;
    for (uint32_t it = 0; ok && c.valid; ++it) {
      const int h = c.seg & 1;
      if (it >= 1) ok = wait_for(a, &ctl->s_free, (it - 1) & 1u);
      if (ok && c.first) ok = wait_for(a, &ctl->q_full[h], (uint32_t)(c.seg >> 1) & 1u);
      if (ok) ok = wait_for(a, &ctl->k_full[rk.s], rk.ph);
      if (!ok) break;
      const uint32_t q0 = qa + ((c.prefix || !halves) ? 0 : h * 8192);
      const uint32_t d = tmem + C::T_S;
      tc::fence_after_sync();
      if (lane == 0) {
        const uint32_t k0 = ra + rk.s * C::STAGE;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_pair(d, tc::sdesc_at(C::DESC_K, q0 + (k >> 2) * 16384 + (k & 3) * 32),
                   tc::sdesc_at(C::DESC_K, k0 + (k >> 2) * 8192 + (k & 3) * 32), C::IDESC_QK, k != 0);
        commit_pair(&ctl->s_full[rk.s]);
        if (c.last) commit_pair(&ctl->q_done[h]);
      }
      __syncwarp();
      rk.step();
      c.next(p);
    }
  } else if (warp == kPvWarp) {
    // ---- outputs, by the first CTA for both ----
    Cursor c;
    c.init(p, ctl);
    Ring<C::NV> rv;
    bool ok = rank == 0;
    const uint32_t ra = base + kCtrlBytes + C::QBYTES + C::NK * C::STAGE;
    const int rpb = a.page < 64 ? a.page : 64, rsh = 31 - __clz(rpb);
    for (uint32_t it = 0; ok && c.valid; ++it) {
      const uint32_t pa = tmem + C::T_P + (it & 1u) * 64, vs = ra + rv.s * C::STAGE;
      const int n = c.count(), steps = (n + 15) >> 4;
      ok = wait_for(a, &ctl->v_full[rv.s], rv.ph);
      if (!ok) break;
      ok = wait_for(a, &ctl->p_ready[it & 1u], (it >> 1) & 1u);
      if (!ok) break;
      tc::fence_after_sync();
      if (lane == 0) {
        const uint64_t dv = desc_v<D>(rpb * C::VROW);
        // keys 16 k ..: pieces of rpb keys with all their blocks, one after the other.
        // (Unrolled: the addresses of a step computed in a loop took longer than its
        // product.)
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          if (k < steps)
            mma_pair_ts(tmem, pa + k * 8,
                        tc::sdesc_at(dv, vs + k * 16 * C::VROW + (((k * 16) >> rsh) << rsh) * (D - C::VROW)),
                        C::IDESC_PV, k == 0 ? !c.first : 1u);
        commit_pair(&ctl->pv_done[rv.s]);
        if (c.last) commit_pair(&ctl->seg_done);
      }
      __syncwarp();
      rv.step();
      c.next(p);
    }
  } else if (warp == kCleanWarp) {
    // ---- values that a row of the job does not see ----
    // The last 16 rows that the product reads: zeros past the end.  Tokens that only
    // some queries of a sequence see: no infinities or NaN.
    Cursor c;
    c.init(p, ctl);
    Ring<C::NV> rv;
    uint32_t phases = 0;      // one bit per stage: its use of `landed` that comes next
    bool ok = true;
    const int rpb = a.page < 64 ? a.page : 64;
    constexpr int chunks = D / 16;   // 16-byte pieces of a row
    for (; c.valid; c.next(p), rv.step()) {
      if (!cleaned<several>(a, c)) continue;
      const int n = c.count();
      ok = wait_for(a, &ctl->landed[rv.s], (phases >> rv.s) & 1u);
      if (!ok) break;
      phases ^= 1u << rv.s;
      uint8_t* const v = ring + (C::NK + rv.s) * C::STAGE;
      const int from = max(c.keys - a.steps + 1 - c.t * kTile, 0);   // the first hidden token
      if (several && !c.prefix && from < n) {
        const bool found = clear_not_finite<D>(v, from, n, rpb);
        // for the join: by CTA, and whether more of the hidden tokens come in the next tile
        if (lane == 0) p.hidden[c.slot_job * 4 + (c.keys - c.t * kTile > kTile ? 2 : 0) + rank] = found;
      }
      for (int w = lane; w < (-n & 15) * chunks; w += 32)
        *v_chunk<D>(v, n + w / chunks, w % chunks, rpb) = make_uint4(0, 0, 0, 0);
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) arrive_at(peer(tc::smem_u32(&ctl->v_full[rv.s]), 0));
    }
  } else {
    // ---- softmax and the share's partial results ----
    Cursor c;
    c.init(p, ctl);
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const float sc = a.scale * 1.44269504088896340736f;   // scores in binary orders
    const int step = row / pl.G;                          // of a tail's row
    uint32_t it = 0, met = 0;
    Ring<C::NK> rs;       // tile it's scores
    Ring<C::NV> ro, rp;   // the O products of tiles it - 1 and it - 2
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    // A finished segment is written out in the next one's first tile, after that
    // tile's weights: its last product runs meanwhile, and the next segment's first
    // product, which overwrites O, waits for the weights' arrival.
    struct {
      bool pending = false;
      uint32_t seg;
      int rows, stride;
      long long row0;
      float m, l;
    } done;
    auto write_out = [&]() {
      done.pending = false;
      ok = wait_for(a, &ctl->seg_done, done.seg & 1u);
      if (!ok || quarter * 32 >= done.rows) return;
      tc::fence_after_sync();
      const bool mine = row < done.rows;
      if (mine) {
        float* w = reinterpret_cast<float*>(p.ml + done.row0 + row);
        if (half == 0) *reinterpret_cast<float2*>(w) = make_float2(done.m, done.l);
        else w[2] = done.l;
      }
      float4* o4 = reinterpret_cast<float4*>(p.opart) + done.row0 * (D / 4) + (long long)(half * (D / 8)) * done.stride + row;
#pragma unroll 1
      for (int o = 0; o < D / 2; o += 32) {
        float v[32];
        tc::tmem_ld32(tmem + lanes + half * (D / 2) + o, v);
        if (mine) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            o4[(long long)j * done.stride] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
        o4 += 8 * (long long)done.stride;
      }
    };
    while (ok && c.valid) {
      // this CTA's rows of the job
      const int rows = c.prefix ? min(max(pl.ntok - (2 * c.mb + (int)rank) * pl.tpb, 0), pl.tpb) * pl.G
                                : (rank == 0 ? pl.R : 0);
      const bool active = quarter * 32 < rows;
      ok = wait_for(a, &ctl->s_full[rs.s], rs.ph);
      if (!ok) break;
      tc::fence_after_sync();
      float s[64];
      if (active) tmem_ld64(tmem + lanes + C::T_S + half * 64, s);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_at(peer(tc::smem_u32(&ctl->s_free), 0));
      // the weights go where those of tile it - 2 were
      if (it >= 2) {
        ok = wait_for(a, &ctl->pv_done[rp.s], rp.ph);
        if (!ok) break;
        tc::fence_after_sync();
        rp.step();
      }
      if (active) {
        // keys this row sees in its half of the tile
        int see = c.keys - c.t * kTile;
        if (!c.prefix) see -= a.steps - 1 - step;
        const int nv = row < rows ? see - half * 64 : 0;
        if (!__all_sync(0xffffffffu, nv >= 64)) {
#pragma unroll
          for (int j = 0; j < 64; ++j) s[j] = j < nv ? s[j] : -INFINITY;
        }
        float mq[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int j = 4; j < 64; ++j) mq[j & 3] = fmaxf(mq[j & 3], s[j]);
        float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
        ctl->red[it & 1u][half][row] = mx;
        __syncwarp();
        if (lane == 0) arrive(&ctl->pair[quarter]);
        ok = wait_for(a, &ctl->pair[quarter], met);
        if (!ok) break;
        met ^= 1u;
        mx = fmaxf(mx, ctl->red[it & 1u][half ^ 1][row]) * sc;
        if (c.first) {
          m = mx;
          l = 0.0f;
        } else {
          const bool grow = mx > m + 8.0f;
          if (__any_sync(0xffffffffu, grow)) {
            // O is behind by 2^8 or more in some row: bring it to the new maximum.
            ok = wait_for(a, &ctl->pv_done[ro.s], ro.ph);
            if (!ok) break;
            tc::fence_after_sync();
            const float f = grow ? ex2(m - mx) : 1.0f;
            if (grow) {
              m = mx;
              l *= f;
            }
#pragma unroll 1
            for (int o = 0; o < D / 2; o += 32) {
              float v[32];
              const uint32_t at = tmem + lanes + half * (D / 2) + o;
              tc::tmem_ld32(at, v);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] *= f;
              tc::tmem_st32(at, v);
            }
          }
        }
        const float mu = finite_base(m);
        float pk[32];
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float e0 = ex2(fmaf(s[2 * j], sc, -mu)), e1 = ex2(fmaf(s[2 * j + 1], sc, -mu));
          s0 += e0;
          s1 += e1;
          pk[j] = __uint_as_float(pack_bf16x2(e0, e1));
        }
        l += s0 + s1;
        tc::tmem_st32(tmem + lanes + C::T_P + (it & 1u) * 64 + half * 32, pk);
      }
      if (done.pending) {
        write_out();
        if (!ok) break;
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_at(peer(tc::smem_u32(&ctl->p_ready[it & 1u]), 0));
      if (c.last) {
        const long long slot = c.slot_job + share;
        // which shares hold the job's ranges, for the join
        if (rank == 0 && warp == 2 && lane == 0) {
          const int job = c.prefix ? c.slot_job : pl.np + c.slot_job;
          if (c.t0 == 0) p.span[job].x = share;
          if ((long long)c.t1 * kTile >= c.keys) p.span[job].y = share;
        }
        done.pending = true;
        done.seg = (uint32_t)c.seg;
        done.rows = rows;
        done.stride = c.prefix ? 128 : pl.R;
        done.row0 = c.prefix ? slot * 256 + rank * 128
                             : (long long)(pl.np ? pl.np + pl.shares : 0) * 256 + slot * pl.R;
        done.m = m;
        done.l = l;
      }
      if (it > 0) ro.step();
      rs.step();
      ++it;
      c.next(p);
    }
    if (ok && done.pending) write_out();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  cluster_sync();   // no product, report or arrival of the other CTA is on its way here any more
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Joins a token's ranges: a CTA takes one query token, one key head and d /
// gridDim.z of its dimensions; a thread one group head and four dimensions of a
// share of the ranges, the shares meeting in shared memory in a fixed order.  (A
// CTA finds its ranges first, at a cost of some trips to L2, so few CTAs with all
// of a head's dimensions each are better than many with 32 as soon as they fill
// the GPU: 25 us of the latter for 512 tokens and heads.)
constexpr int kJoinThreads = 256;

// (Of several query tokens a sequence the first kernel leaves out what is not finite
// in the last ones' values.)
template <int D, bool several>
__global__ void __launch_bounds__(kJoinThreads) attn_shared_join(const __grid_constant__ SharedParams p) {
  __shared__ float4 acc[kJoinThreads];
  __shared__ float2 stat[kJoinThreads];
  const AttnSharedArgs& a = p.a;
  const Plan& pl = p.pl;
  const int tok = blockIdx.x, hk = blockIdx.y, width4 = D / 4 / gridDim.z;   // in groups of 4 dimensions
  const int b = tok / a.steps, step = tok - b * a.steps;
  // this token's two jobs for this key head, its prefix block and its tail: a range in
  // share c has slot job + c
  const int blk = tok / pl.tpb;                            // block of a CTA's rows
  const int job[2] = {hk * pl.nmb + (blk >> 1), b * pl.h_kv + hk};
  const int stride[2] = {128, pl.R};                       // rows of a CTA's part of a slot
  const int in[2] = {(tok - blk * pl.tpb) * pl.G, step * pl.G};
  const int apart[2] = {256, pl.R};                        // slots are so many rows apart
  // Launched while the first kernel runs; its results are there from here on.  (The
  // next call's kernel is not let begin before this one ends: its CTAs then took the
  // SMs as they fell free, 176 us a call for 169 at 256 sequences.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 none = make_int2(0, -1);   // no range
  const int2 pre_at = pl.np ? p.span[job[0]] : none;
  const int2 own_at = a.tail_width > 0 && a.tail_len[b] > 0 ? p.span[pl.np + job[1]] : none;
  const Ranges pre = ranges_of(pre_at.x, pre_at.y, pl.shares), own = ranges_of(own_at.x, own_at.y, pl.shares);
  const long long first[2] = {
      (long long)(job[0] + pre.first) * 256 + (blk & 1) * 128,
      (long long)(pl.np ? pl.np + pl.shares : 0) * 256 + (long long)(job[1] + own.first) * pl.R};

  // The tokens that this one sees and some other query of its sequence does not: [from,
  // see), none unless the first kernel left something out among them.
  int from = 0, see = 0;
  if (several) {
    const int len = tail_length(a, b);
    const uchar4 found = *reinterpret_cast<const uchar4*>(p.hidden + job[1] * 4);
    from = max(len - a.steps + 1, 0);
    if (len > 0 && (found.x | found.y | (from / kTile < (len - 1) / kTile ? found.z | found.w : 0)) != 0)
      see = len - (a.steps - 1 - step);
  }

  const int items = pl.G * width4, d0 = blockIdx.z * width4;
  for (int i0 = 0; i0 < items; i0 += kJoinThreads) {
    const int width = min(items - i0, kJoinThreads), groups = kJoinThreads / width;
    const int grp = threadIdx.x / width, item = i0 + threadIdx.x % width;
    const int c4 = d0 + item / pl.G, g = item % pl.G;
    float M = -INFINITY, L = 0.0f;
    float4 o = make_float4(0, 0, 0, 0);
    const int h = hk * pl.G + g;
    uint2 gt = make_uint2(0, 0);
    if (a.gate && threadIdx.x < width)   // on its way under the sums
      gt = *reinterpret_cast<const uint2*>(a.gate + tok * a.gate_st + h * a.gate_sh + 4 * c4);
    if (grp < groups) {
      // a job's ranges, four at a time: their loads are all in flight before the first
      // is added
      const auto join = [&](const float4* ml, const float4* v, int n, long long ml_step, long long v_step) {
        for (int i = grp; i < n; i += 4 * groups) {
          float4 mv[4], vv[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = i + u * groups;
            mv[u] = r < n ? ml[r * ml_step] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
            vv[u] = r < n ? v[r * v_step] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          }
          // Only a range with a sum counts (one without saw no key).  A NaN sum counts,
          // though its maximum may be NaN or -inf (fmaxf drops NaN): the row is NaN then.
          float mn = M, sum[4];
          bool any = false;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            sum[u] = mv[u].y + mv[u].z;
            any |= sum[u] != 0.0f;
            if (sum[u] != 0.0f) mn = fmaxf(mn, mv[u].x);
          }
          if (!any) continue;   // rows that see nothing so far
          const float base = finite_base(mn), f = ex2(M - base);
          L *= f;
          o.x *= f;
          o.y *= f;
          o.z *= f;
          o.w *= f;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (sum[u] == 0.0f) continue;
            const float w = ex2(mv[u].x - base);
            L += sum[u] * w;
            o.x += vv[u].x * w;
            o.y += vv[u].y * w;
            o.z += vv[u].z * w;
            o.w += vv[u].w * w;
          }
          M = mn;
        }
      };
      const float4* part = reinterpret_cast<const float4*>(p.opart);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        join(p.ml + first[k] + in[k] + g, part + first[k] * (D / 4) + (long long)c4 * stride[k] + in[k] + g,
             k ? own.count : pre.count, apart[k], (long long)apart[k] * (D / 4));
    }
    acc[threadIdx.x] = o;
    stat[threadIdx.x] = make_float2(M, L);
    __syncthreads();
    if (threadIdx.x < width) {
      for (int q = 1; q < groups; ++q) {
        const float2 st = stat[q * width + threadIdx.x];
        const float4 v = acc[q * width + threadIdx.x];
        if (st.y == 0.0f) continue;
        const float mn = fmaxf(M, st.x), base = finite_base(mn);
        const float f = ex2(M - base), w = ex2(st.x - base);
        L = L * f + st.y * w;
        o.x = o.x * f + v.x * w;
        o.y = o.y * f + v.y * w;
        o.z = o.z * f + v.z * w;
        o.w = o.w * f + v.w * w;
        M = mn;
      }
      // no key seen: zeros.  (A NaN sum stays NaN.)
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      float r[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
      if (several) {
#pragma unroll 1
        for (int j = from; j < see; ++j) {
          const int pg = a.tail_pages[(size_t)b * a.tail_width + j / a.page];
          if (pg < 0 || pg >= a.n_pages) continue;
          const size_t at = ((size_t)pg * a.page + j % a.page) * pl.h_kv + hk;
          const uint2 v = *reinterpret_cast<const uint2*>(a.v_cache + at * D + 4 * c4);
          const uint32_t x = not_finite(v.x), y = not_finite(v.y);
          r[0] += __uint_as_float(x << 16);
          r[1] += __uint_as_float(x & 0xffff0000u);
          r[2] += __uint_as_float(y << 16);
          r[3] += __uint_as_float(y & 0xffff0000u);
        }
      }
      if (a.gate) {
        r[0] *= sigmoid(__uint_as_float(gt.x << 16));
        r[1] *= sigmoid(__uint_as_float(gt.x & 0xffff0000u));
        r[2] *= sigmoid(__uint_as_float(gt.y << 16));
        r[3] *= sigmoid(__uint_as_float(gt.y & 0xffff0000u));
      }
      uint2 w;
      w.x = pack_bf16x2(r[0], r[1]);
      w.y = pack_bf16x2(r[2], r[3]);
      *reinterpret_cast<uint2*>(a.out + ((long long)tok * a.h_q + h) * D + 4 * c4) = w;
    }
    __syncthreads();
  }
}

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
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

bool encode(CUtensorMap* m, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
  if (!enc) return false;
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The cache as [block of 64 dimensions][token row][64 dimensions].  K: boxes of a
// page piece with all of a head's blocks when the piece is 64 rows, else with one
// block.  V: boxes of a page piece with half of a head's dimensions.
bool cache_map(CUtensorMap* m, const AttnSharedArgs& p, const void* base, bool v) {
  const cuuint32_t rpb = p.page < 64 ? p.page : 64;
  const cuuint64_t dims[3] = {64, (cuuint64_t)p.n_pages * p.page, (cuuint64_t)p.h_kv * p.d / 64};
  const cuuint64_t strides[2] = {(cuuint64_t)p.h_kv * p.d * 2, 128};
  const cuuint32_t blocks = v ? (p.d == 64 ? 1 : p.d / 128) : (rpb == 64 ? p.d / 64 : 1);
  const cuuint32_t box[3] = {v && p.d == 64 ? 32u : 64u, rpb, blocks};
  return encode(m, base, dims, strides, box, v && p.d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// q as [token][head][d]: boxes of 64 dimensions by a group's heads by `tokens` tokens.
bool q_map(CUtensorMap* m, const AttnSharedArgs& p, int G, int tokens) {
  const cuuint64_t dims[3] = {(cuuint64_t)p.d, (cuuint64_t)p.h_q, (cuuint64_t)p.batch * p.steps};
  const cuuint64_t strides[2] = {(cuuint64_t)p.d * 2, (cuuint64_t)p.h_q * p.d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)tokens};
  return encode(m, p.q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

Plan make_plan(int batch, int steps, int h_q, int h_kv, long long prefix_len, int shares) {
  Plan pl;
  pl.h_kv = h_kv;
  pl.G = h_q / h_kv;
  pl.R = steps * pl.G;
  pl.ntok = batch * steps;
  pl.tpb = 128 / pl.G;
  pl.nmb = (pl.ntok + 2 * pl.tpb - 1) / (2 * pl.tpb);
  pl.ptiles = (prefix_len + kTile - 1) / kTile;
  pl.np = pl.ptiles > 0 ? h_kv * pl.nmb : 0;
  pl.shares = shares;
  pl.wp = pl.np * (pl.ptiles * kCostPrefix + kCostJob);
  return pl;
}

// Slot rows: a job's range in share c has slot job + c (each step to the next
// range moves to the next job, the next share or both).
size_t slot_rows(const Plan& pl, int batch) {
  return (size_t)(pl.np ? pl.np + pl.shares : 0) * 256 + ((size_t)batch * pl.h_kv + pl.shares) * pl.R;
}

template <int D>
cudaError_t launch_d(const AttnSharedArgs& a, cudaStream_t stream, int sms) {
  using C = Cfg<D>;
  SharedParams p;
  p.a = a;
  p.pl = make_plan(a.batch, a.steps, a.h_q, a.h_kv, a.prefix_len,
                   sms < 2 ? 1 : (sms / 2 < kMaxShares ? sms / 2 : kMaxShares));
  char* ws = static_cast<char*>(a.scratch);
  p.span = reinterpret_cast<int2*>(ws);
  ws += up256(((size_t)p.pl.np + (size_t)a.batch * a.h_kv) * sizeof(int2));
  p.hidden = reinterpret_cast<uint8_t*>(ws);
  ws += up256((size_t)a.batch * a.h_kv * 4);
  const size_t rows = slot_rows(p.pl, a.batch);
  p.ml = reinterpret_cast<float4*>(ws);
  ws += up256(rows * sizeof(float4));
  p.opart = reinterpret_cast<float*>(ws);

  CUtensorMap tk, tv, tqp, tqt;
  const bool cached = a.prefix_len > 0 || a.tail_width > 0;
  // without a cache no tile is loaded; q stands in for the unused maps
  if (!q_map(&tqp, a, p.pl.G, p.pl.tpb) || !q_map(&tqt, a, p.pl.G, a.steps)) return cudaErrorInvalidValue;
  tk = tv = tqp;
  if (cached && (!cache_map(&tk, a, a.k_cache, false) || !cache_map(&tv, a, a.v_cache, true))) return cudaErrorInvalidValue;
  cudaError_t e;
  const auto kernel = a.steps > 1 ? attn_shared_kernel<D, true> : attn_shared_kernel<D, false>;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)C::SMEM)) != cudaSuccess)
    return e;
  // each launch passes under the kernel before it
  cudaLaunchAttribute overlap;
  overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  overlap.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.pl.shares);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kernel, tk, tv, tqp, tqt, p)) != cudaSuccess) return e;
  int nz = 1;   // CTAs per token and key head
  while (nz < D / 32 && (long long)p.pl.ntok * p.pl.h_kv * nz < 6LL * sms) nz *= 2;
  cfg.gridDim = dim3(p.pl.ntok, p.pl.h_kv, nz);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, a.steps > 1 ? attn_shared_join<D, true> : attn_shared_join<D, false>, p);
}

}  // namespace

size_t attn_shared_scratch_bytes(int batch, int steps, int h_q, int h_kv, int d) {
  const Plan pl = make_plan(batch > 0 ? batch : 1, steps, h_q, h_kv, 1, kMaxShares);
  const size_t rows = slot_rows(pl, batch);
  return up256(((size_t)pl.np + (size_t)batch * h_kv) * sizeof(int2)) + up256((size_t)batch * h_kv * 4) +
         up256(rows * sizeof(float4)) + up256(rows * d * 4);
}

cudaError_t launch_attn_shared(const AttnSharedArgs& p, cudaStream_t stream) {
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
