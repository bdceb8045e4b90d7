// gdn_pages.cu -- the pool that cache pages come from: sequences growing, trimmed, forked
// and freed, the pool drawn together, pages copied (gdn_pages_*).
//
// Integers first.  A call looks at its whole list before it changes anything, so that it
// is done whole or not at all, and pages are handed out lowest first, in the list's order:
// results follow from the arguments alone.  That needs sums over the list and over the
// pool's counts, with every part of the pool seen before the first change: one cluster of
// eight CTAs does it in one launch, its barrier standing between the looking and the
// changing.  (A grid-wide barrier or a second launch costs more than eight SMs take for
// the counts of 65536 pages.)  Every CTA sums the list by itself, which spares a barrier;
// the pool's counts are looked through 65536 at a time, until enough free pages are found.
//
// Bytes then.  Whole pages move by a second kernel over the whole GPU, a warp 4 KB at a time
// with eight 16-byte loads in flight per lane before the first store; it finds how many
// there are in the workspace, and also changes the tables where there is much of them.
//
// Measured: 4 tokens more for 256 sequences in a pool of 65536 pages 5.5 us (lists and counts
// loaded 1.4, sums 0.7, free pages shared out 1.9, rows and tables written 1.3), taking them back
// 3.8; forking 48 children of 5003 tokens with 12 caches of 36 KB pages 5.8 + 6 us; drawing
// 6656 pages of 12 caches together, 3482 of them in use and some 1660 to be moved, 224 us, 6.6 TB/s
// read and written, 98 % of a copy's rate.
#include <limits.h>

#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

constexpr int kCluster = 8;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMoveWarps = 8;
constexpr int kMoveBytes = 32 * 16 * 8;   // of a page that a warp moves at a time

// Workspace: a header, then lists of n_pages entries each.
struct Header {
  int moves;       // page pairs to copy; 0 too where the call does nothing
  int live;        // pages in use after a compaction
  int pairs;       // forked pairs
};

struct PoolParams {
  PagePool pool;
  const int32_t *seq, *to, *arg;   // list; fork's destinations; counts or new lengths
  int32_t *slot, *n_live;
  int32_t* status;
  Header* head;
  int32_t *from, *dest;            // [n_pages] pairs of the copies; dest holds the free pages found
  int32_t* remap;                  // [n_pages] new places of pages, or
  int2* pair;                      // [list] (length, new last page or -1) of a fork
  int n, steps;
};

enum Op { kExtend, kTrim, kFork, kFree };

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

// v into the same place of shared memory of CTA `rank`.
__device__ __forceinline__ void store_to(int* at, uint32_t rank, int v) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(at)), b;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(b), "r"(v) : "memory");
}

template <typename T>
__device__ __forceinline__ T warp_scan(T v) {   // inclusive
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const T o = __shfl_up_sync(0xffffffffu, v, m);
    if (threadIdx.x % 32 >= m) v += o;
  }
  return v;
}

// What the threads before this one have in all, and the CTA's total.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* warp_sums, T& total) {
  static_assert(kPlanWarps == 32, "the warps' sums are one to a lane");
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const T s = warp_scan(v);
  __syncthreads();                          // the sums of a scan before may still be read
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  const T all = warp_scan(warp_sums[lane]);
  total = __shfl_sync(0xffffffffu, all, 31);
  const T before = __shfl_sync(0xffffffffu, all, warp == 0 ? 0 : warp - 1);
  return (warp == 0 ? 0 : before) + s - v;
}

struct Shared {
  uint32_t seen[GDN_PAGES_MAX_SEQS / 32];
  long long need_sums[kPlanWarps];
  int free_sums[kPlanWarps];
  int found[2][kCluster];
  uint16_t mine[8 * kPlanThreads];   // this CTA's free pages of the first tile
};

// Four counts from page 4 i on; past the pool's end they read as in use.
__device__ __forceinline__ int4 counts(const PagePool& p, int i) {
  if (4LL * i + 3 < p.n_pages) return *reinterpret_cast<const int4*>(p.refs + 4LL * i);
  int4 c = make_int4(1, 1, 1, 1);
  if (4LL * i < p.n_pages) c.x = p.refs[4LL * i];
  if (4LL * i + 1 < p.n_pages) c.y = p.refs[4LL * i + 1];
  if (4LL * i + 2 < p.n_pages) c.z = p.refs[4LL * i + 2];
  return c;
}

// Which of this thread's eight pages of a tile (65536 pages, over the cluster) are free.
__device__ __forceinline__ uint32_t free_pages(const PagePool& p, int tile) {
  const int at = tile + ((int)cluster_rank() * kPlanThreads + (int)threadIdx.x) * 2;
  const int4 c = counts(p, at), d = counts(p, at + 1);
  return (c.x <= 0) | (c.y <= 0) << 1 | (c.z <= 0) << 2 | (c.w <= 0) << 3 | (d.x <= 0) << 4 | (d.y <= 0) << 5 |
         (d.z <= 0) << 6 | (d.w <= 0) << 7;
}
constexpr int kTileGroups = kCluster * kPlanThreads * 2;   // groups of four pages of a tile

// Hands out the lowest `need` free pages: give(k, page) for the k-th of them, by whichever thread
// of the cluster, once every CTA is here and only where there are as many; false where not.  Of
// the first tile the caller has this thread's pages in `mask`, the free ones in the threads
// before it in `before` and the CTA's in `total`.  Where the first tile holds enough, each CTA
// gives the pages that it found, a thread each (they often lie together); else all go through
// list[] first.
template <typename Give>
__device__ __forceinline__ bool hand_out(const PagePool& p, long long need, uint32_t mask, int before, int total,
                                         int32_t* list, Shared& sh, const Give& give) {
  const int rank = (int)cluster_rank();
  if (need == 0) {
    cluster_sync();
    return true;
  }
  long long have = 0;
  for (int tile = 0, turn = 0; have < need && (long long)tile * 4 < p.n_pages; tile += kTileGroups, turn ^= 1) {
    if (tile > 0) {
      mask = free_pages(p, tile);
      before = block_scan(__popc(mask), sh.free_sums, total);
    }
    if (threadIdx.x < kCluster) store_to(&sh.found[turn][rank], threadIdx.x, total);
    cluster_sync();
    long long base = have;                       // free pages before this CTA's
    for (int r = 0; r < kCluster; ++r) {
      base += r < rank ? sh.found[turn][r] : 0;
      have += sh.found[turn][r];
    }
    const int first = 4 * (tile + rank * kPlanThreads * 2);   // this CTA's first page
    if (tile == 0 && have >= need) {
      int at = before;
      for (uint32_t m = mask; m != 0 && base + at < need; m &= m - 1, ++at)
        sh.mine[at] = (uint16_t)(threadIdx.x * 8 + __ffs(m) - 1);
      __syncthreads();
      for (int k = threadIdx.x; k < total && base + k < need; k += kPlanThreads) give((int)base + k, first + sh.mine[k]);
      return true;
    }
    long long at = base + before;
    for (uint32_t m = mask; m != 0 && at < need; m &= m - 1, ++at) list[at] = first + (int)threadIdx.x * 8 + __ffs(m) - 1;
  }
  cluster_sync();
  if (have < need) return false;
  for (int k = rank * kPlanThreads + (int)threadIdx.x; k < need; k += kCluster * kPlanThreads) give(k, list[k]);
  return true;
}

__device__ __forceinline__ bool in_pool(const PagePool& p, int page) { return page >= 0 && page < p.n_pages; }

__device__ __forceinline__ int pages_of(const PagePool& p, int tokens) { return (int)(((long long)tokens + p.page - 1) / p.page); }

// Item i of the list: its sequence, tokens and the new pages it needs; false if it may not be.
template <Op OP>
__device__ __forceinline__ bool look(const PoolParams& a, int i, Shared& sh, int& len, int& need) {
  const PagePool& p = a.pool;
  const long long most = (long long)p.width * p.page;
  const int s = a.seq ? a.seq[i] : i;
  len = need = 0;
  if (s < 0 || s >= p.n_seqs) return false;
  const int changed = OP == kFork ? a.to[i] : s;   // no sequence may be changed twice
  if (changed < 0 || changed >= p.n_seqs) return false;
  if ((OP == kFork || a.seq) && (atomicOr(&sh.seen[changed / 32], 1u << (changed % 32)) >> (changed % 32) & 1)) return false;
  len = p.len[s];
  if (len < 0 || len > most) return false;
  const int32_t* row = p.table + (long long)s * p.width;
  if (OP == kExtend) {
    const int c = a.arg ? a.arg[i] : a.steps;
    if (c < 0 || c > a.steps || (long long)len + c > most) return false;
    need = pages_of(p, len + c) - pages_of(p, len);
  } else if (OP == kTrim) {
    const int to = a.arg[i];
    if (to < 0 || to > len) return false;
    if (to < len && to % p.page != 0) {            // it will end inside a page that others may hold too
      const int e = row[to / p.page];
      need = in_pool(p, e) && p.refs[e] > 1 ? 1 : 0;
    }
  } else if (OP == kFork) {
    if (p.len[changed] != 0) return false;
    need = len % p.page != 0 ? 1 : 0;
  }
  return true;
}

template <Op OP>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads, 1) pages_plan_kernel(PoolParams a) {
  __shared__ Shared sh;
  extern __shared__ int list[];                    // [n + 1] new pages before item i, [n] its tokens
  cluster_arrive();                                // waited for before shared memory of another CTA is written
  int *off = list, *len0 = list + a.n + 1;
  const PagePool& p = a.pool;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int rank = (int)cluster_rank(), thread = rank * kPlanThreads + (int)threadIdx.x;
  for (int i = threadIdx.x; i < GDN_PAGES_MAX_SEQS / 32; i += kPlanThreads) sh.seen[i] = 0;
  __syncthreads();
  // the list, by every CTA, and under its loads those of the pool's first tile (of a trim or a
  // free, which hardly ever or never need a page, only where they do)
  uint32_t mask = OP == kExtend || OP == kFork ? free_pages(p, 0) : 0;
  const int per = (a.n + kPlanThreads - 1) / kPlanThreads, i0 = threadIdx.x * per;
  long long mine = 0;
  bool good = true;
  for (int i = i0; i < min(i0 + per, a.n); ++i) {
    int need;
    good = look<OP>(a, i, sh, len0[i], need) && good;
    off[i] = need;
    mine += need;
  }
  // (a trim or a free as a rule needs no page: its sums are spared)
  long long total = 0, at = 0;
  if (OP == kExtend || OP == kFork || __syncthreads_or(mine != 0)) at = block_scan(mine, sh.need_sums, total);
  for (int i = i0; i < min(i0 + per, a.n); ++i) {
    const int need = off[i];
    off[i] = (int)at;
    at += need;
  }
  if (threadIdx.x == 0) off[a.n] = (int)total;
  if ((OP == kTrim || OP == kFree) && total > 0) mask = free_pages(p, 0);
  int before = 0, here = 0;
  if (total > 0) before = block_scan(__popc(mask), sh.free_sums, here);
  bool ok = __syncthreads_and(good) && total <= p.n_pages;
  cluster_wait();
  // Every CTA came to the same ok; no CTA gets past hand_out's first barrier, behind which the
  // changes are, before all have looked at everything.
  const auto give = [&](int k, int page) {
    int lo = 0, hi = a.n;                          // the item it goes to: the last with off[lo] <= k
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (off[mid] <= k) lo = mid; else hi = mid;
    }
    const int s = a.seq ? a.seq[lo] : lo, len = len0[lo];
    int32_t* row = p.table + (long long)s * p.width;
    if (OP == kExtend) {
      const int col = pages_of(p, len) + k - off[lo], count = a.arg ? a.arg[lo] : a.steps;
      row[col] = page;
      p.refs[page] = 1;
      const int end = min((col + 1LL) * p.page, (long long)len + count) - (long long)col * p.page;
      int32_t* slot = a.slot + (long long)lo * a.steps + (col * p.page - len);
      for (int j = 0; j < end; ++j) slot[j] = page * p.page + j;
    } else if (OP == kFork) {
      a.from[k] = row[len / p.page];
      a.dest[k] = page;
      a.pair[lo] = make_int2(len, page);
    } else if (OP == kTrim) {
      const int col = a.arg[lo] / p.page, old = row[col];
      row[col] = page;
      p.refs[page] = 1;
      atomicSub(p.refs + old, 1);
      a.from[k] = old;
      a.dest[k] = page;
    }
  };
  ok = hand_out(p, ok ? total : 0, mask, before, here, a.dest, sh, give) && ok;
  if (!ok) {
    if (thread == 0) record_status(a.status, GDN_ERR_DEVICE_BOUNDS);
    if (thread == 0 && OP != kExtend && OP != kFree) a.head->moves = a.head->pairs = 0;
    if (OP == kExtend)
      for (long long x = thread; x < (long long)a.n * a.steps; x += kCluster * kPlanThreads) a.slot[x] = -1;
  } else if (OP == kExtend) {
    // rows of pages that were there already, and none
    const long long slots = (long long)a.n * a.steps;
    for (long long x = thread; x < slots; x += kCluster * kPlanThreads) {
      const int i = slots <= INT_MAX ? (int)x / a.steps : (int)(x / a.steps), st = (int)(x - (long long)i * a.steps);
      const int s = a.seq ? a.seq[i] : i, c = a.arg ? a.arg[i] : a.steps, len = len0[i];
      if (st == 0) p.len[s] = len + c;
      const int pos = st < c ? len + st : 0, col = pos / p.page;
      if (st >= c) {
        a.slot[x] = -1;
      } else if (col < pages_of(p, len)) {
        const int page = p.table[(long long)s * p.width + col];
        if (!in_pool(p, page)) record_status(a.status, GDN_ERR_DEVICE_BOUNDS);
        a.slot[x] = in_pool(p, page) ? page * p.page + pos % p.page : -1;
      }
    }
  } else if (OP == kFork) {
    if (thread == 0) {
      a.head->moves = (int)total;
      a.head->pairs = a.n;
    }
    for (int i = thread; i < a.n; i += kCluster * kPlanThreads)
      if (off[i + 1] == off[i]) a.pair[i] = make_int2(len0[i], -1);
  } else {                                         // trim and free: a warp per sequence
    if (OP == kTrim && thread == 0) {
      a.head->moves = (int)total;
      a.head->pairs = 0;
    }
    const int lane = threadIdx.x % 32;
    for (int i = thread / 32; i < a.n; i += kCluster * kPlanWarps) {
      const int s = a.seq ? a.seq[i] : i, to = OP == kTrim ? a.arg[i] : 0;
      int32_t* row = p.table + (long long)s * p.width;
      const int had = pages_of(p, len0[i]);
      for (int col = pages_of(p, to) + lane; col < had; col += 32) {
        const int e = row[col];
        if (in_pool(p, e)) atomicSub(p.refs + e, 1);
        else record_status(a.status, GDN_ERR_DEVICE_BOUNDS);
        row[col] = -1;
      }
      if (lane == 0) p.len[s] = to;
    }
  }
  if (OP == kFork || OP == kTrim) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Compaction: with n_live pages in use, the i-th free page below n_live takes what the i-th
// page in use at or above it holds.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads, 1) pages_compact_kernel(PoolParams a) {
  __shared__ Shared sh;
  cluster_arrive();                                // as above
  const PagePool& p = a.pool;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int rank = (int)cluster_rank(), thread = rank * kPlanThreads + (int)threadIdx.x;
  // each CTA a stretch of the pool, in groups of four pages
  const int groups = (int)(((long long)p.n_pages + 3) / 4), per = (groups + kCluster - 1) / kCluster;
  const int lo = min(rank * per, groups), hi = min(lo + per, groups);
  const auto used = [&](int i) -> uint32_t {       // of four pages; past the pool's end: none
    int4 c = counts(p, i);
    if (4LL * i + 3 >= p.n_pages) {
      c.w = 0;
      if (4LL * i + 2 >= p.n_pages) c.z = 0;
      if (4LL * i + 1 >= p.n_pages) c.y = 0;
    }
    return (c.x > 0) | (c.y > 0) << 1 | (c.z > 0) << 2 | (c.w > 0) << 3;
  };
  int n = 0;
  for (int i = lo + threadIdx.x; i < hi; i += kPlanThreads) n += __popc(used(i));
  int total;
  block_scan(n, sh.free_sums, total);
  cluster_wait();
  if (threadIdx.x < kCluster) store_to(&sh.found[0][rank], threadIdx.x, total);
  cluster_sync();
  int live = 0, before = 0;                        // pages in use in all, and before this stretch
  for (int r = 0; r < kCluster; ++r) {
    before += r < rank ? sh.found[0][r] : 0;
    live += sh.found[0][r];
  }
  // A hole's place in its list: free pages before it.  A late page's: pages in use before
  // it, less those below n_live, which are n_live less the holes; so both need `holes`,
  // the free pages below n_live.  Counted in this stretch and then over the cluster.
  n = 0;
  for (int i = lo + threadIdx.x; i < hi; i += kPlanThreads) {
    const uint32_t below = 4LL * i + 3 < live ? 15u : 4LL * i >= live ? 0u : (1u << (live - 4 * i)) - 1;
    n += __popc(~used(i) & below);
  }
  block_scan(n, sh.free_sums, total);
  if (threadIdx.x < kCluster) store_to(&sh.found[1][rank], threadIdx.x, total);
  cluster_sync();
  int holes = 0;
  for (int r = 0; r < kCluster; ++r) holes += sh.found[1][r];
  for (int tile = lo; tile < hi; tile += kPlanThreads) {
    const int i = tile + (int)threadIdx.x;
    const uint32_t u = i < hi ? used(i) : 0;
    int in_use = before + block_scan(__popc(u), sh.free_sums, total);
    before += total;
    if (i < hi) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int page = 4 * i + k;
        if (page >= p.n_pages) break;
        if (page < live) {
          if (!(u >> k & 1)) a.dest[page - in_use] = page;
        } else if (u >> k & 1) {
          a.from[in_use - (live - holes)] = page;
        } else {
          a.remap[page] = -1;
        }
        in_use += u >> k & 1;
      }
    }
  }
  cluster_sync();
  for (int k = thread; k < holes; k += kCluster * kPlanThreads) {
    const int from = a.from[k], to = a.dest[k];
    a.remap[from] = to;
    p.refs[to] = p.refs[from];
    p.refs[from] = 0;
  }
  if (thread == 0) {
    a.head->moves = holes;
    a.head->live = live;
    a.head->pairs = 0;
    if (a.n_live) *a.n_live = live;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// A fork's rows of the table, a warp per pair.
__device__ void fork_rows(const PoolParams& a) {
  const PagePool& p = a.pool;
  const int lane = threadIdx.x % 32, warp = blockIdx.x * kMoveWarps + threadIdx.x / 32;
  const int pairs = a.head->pairs;
  for (int i = warp; i < pairs; i += gridDim.x * kMoveWarps) {
    const int2 what = a.pair[i];
    const int32_t* src = p.table + (long long)a.seq[i] * p.width;
    int32_t* dst = p.table + (long long)a.to[i] * p.width;
    const int whole = what.x / p.page;
    for (int col = lane; col < whole; col += 32) {
      const int e = src[col];
      dst[col] = e;
      if (in_pool(p, e)) atomicAdd(p.refs + e, 1);
      else record_status(a.status, GDN_ERR_DEVICE_BOUNDS);
    }
    if (lane == 0) {
      p.len[a.to[i]] = what.x;
      if (what.y >= 0) {
        dst[whole] = what.y;
        p.refs[what.y] = 1;
      }
    }
  }
}

// A compaction's new entries, a warp per sequence.
__device__ void remap_rows(const PoolParams& a) {
  const PagePool& p = a.pool;
  const int lane = threadIdx.x % 32, warp = blockIdx.x * kMoveWarps + threadIdx.x / 32;
  const int live = a.head->live;
  for (int s = warp; s < p.n_seqs; s += gridDim.x * kMoveWarps) {
    const int len = p.len[s];
    const bool sound = len >= 0 && len <= (long long)p.width * p.page;
    if (!sound && lane == 0) record_status(a.status, GDN_ERR_DEVICE_BOUNDS);
    int32_t* row = p.table + (long long)s * p.width;
    for (int col = lane; sound && col < pages_of(p, len); col += 32) {
      const int e = row[col];
      const int to = !in_pool(p, e) ? -1 : e < live ? e : a.remap[e];
      if (to < 0) record_status(a.status, GDN_ERR_DEVICE_BOUNDS);
      else if (to != e) row[col] = to;
    }
  }
}

struct MoveParams {
  PageMoves m;
  const Header* head;        // where the pairs' count is; null: m.n
};

// Page pairs of all caches, a warp kMoveBytes at a time.
__device__ __forceinline__ void move_pages(const MoveParams& v) {
  const int lane = threadIdx.x % 32;
  const int n = v.head ? v.head->moves : v.m.n, pieces = v.m.first[v.m.caches];
  const long long items = (long long)n * pieces;
  for (long long x = (long long)blockIdx.x * kMoveWarps + threadIdx.x / 32; x < items;
       x += (long long)gridDim.x * kMoveWarps) {
    const int i = (int)(x / pieces), piece = (int)(x - (long long)i * pieces);
    const int from = v.m.from ? v.m.from[i] : i, to = v.m.to ? v.m.to[i] : i;
    if (from < 0 || from >= v.m.src_pages || to < 0 || to >= v.m.dst_pages) {
      if (lane == 0 && piece == 0) record_status(v.m.status, GDN_ERR_DEVICE_BOUNDS);
      continue;
    }
    int c = 0, hi = v.m.caches;                    // the last cache whose pieces begin at or before this one
    while (hi - c > 1) {
      const int mid = (c + hi) / 2;
      if (v.m.first[mid] <= piece) c = mid; else hi = mid;
    }
    const long long bytes = v.m.bytes[c], at = (long long)(piece - v.m.first[c]) * kMoveBytes + lane * 16;
    const uint8_t* s = v.m.src[c] + (long long)from * bytes;
    uint8_t* d = v.m.dst[c] + (long long)to * bytes;
    uint4 r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (at + k * 512 < bytes) r[k] = *reinterpret_cast<const uint4*>(s + at + k * 512);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (at + k * 512 < bytes) *reinterpret_cast<uint4*>(d + at + k * 512) = r[k];
  }
}

enum Rows { kNoRows, kForkRows, kRemapRows };

template <Rows ROWS>
__global__ void __launch_bounds__(kMoveWarps * 32) pages_move_kernel(const __grid_constant__ PoolParams a,
                                                                     const __grid_constant__ MoveParams v) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (ROWS == kForkRows) fork_rows(a);
  if (ROWS == kRemapRows) remap_rows(a);
  move_pages(v);
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

PoolParams params_of(const PagePool& p, void* scratch) {
  PoolParams a = {};
  a.pool = p;
  char* ws = static_cast<char*>(scratch);
  const size_t list = up256((size_t)p.n_pages * sizeof(int32_t));
  a.head = reinterpret_cast<Header*>(ws);
  a.from = reinterpret_cast<int32_t*>(ws + 256);
  a.dest = reinterpret_cast<int32_t*>(ws + 256 + list);
  a.remap = reinterpret_cast<int32_t*>(ws + 256 + 2 * list);
  a.pair = reinterpret_cast<int2*>(ws + 256 + 3 * list);
  return a;
}

struct Launch {
  cudaLaunchAttribute overlap;
  cudaLaunchConfig_t cfg;
  Launch(unsigned grid, unsigned threads, size_t smem, cudaStream_t stream) : cfg{} {
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &overlap;
    cfg.numAttrs = 1;
  }
};

template <Op OP>
cudaError_t launch_plan(const PoolParams& a, cudaStream_t stream) {
  const size_t smem = (2 * (size_t)a.n + 1) * sizeof(int);
  if (smem + sizeof(Shared) > 48 * 1024) {   // more than a kernel may have unasked
    const cudaError_t e = cudaFuncSetAttribute(pages_plan_kernel<OP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (2 * GDN_PAGES_MAX_LIST + 1) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
  }
  Launch l(kCluster, kPlanThreads, smem, stream);
  return cudaLaunchKernelEx(&l.cfg, pages_plan_kernel<OP>, a);
}

cudaError_t sm_count(int& sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
}

template <Rows ROWS>
cudaError_t launch_moves(const PoolParams& a, const MoveParams& v, long long most, cudaStream_t stream) {
  int sms;
  const cudaError_t e = sm_count(sms);
  if (e != cudaSuccess) return e;
  // Enough warps for every piece there can be, up to sixteen times as many as fit on the GPU:
  // 1660 pages of 12 caches of 36 KB took 242 us with twice as many, whose shares end far
  // apart, and 224 so (9700 CTAs without anything to do cost 1 us).
  const long long want = (most + kMoveWarps - 1) / kMoveWarps, fit = (long long)sms * 64;
  Launch l((unsigned)(want < 1 ? 1 : want < fit ? want : fit), kMoveWarps * 32, 0, stream);
  return cudaLaunchKernelEx(&l.cfg, pages_move_kernel<ROWS>, a, v);
}

MoveParams moves_of(const PoolParams& a, const PageMoves* caches) {
  MoveParams v = {};
  if (caches) v.m = *caches;
  v.m.from = a.from;
  v.m.to = a.dest;
  v.m.src_pages = v.m.dst_pages = a.pool.n_pages;
  v.m.status = a.status;
  v.head = a.head;
  return v;
}

}  // namespace

size_t pages_scratch_bytes(int n_pages, int n_seqs) {
  return 256 + 3 * up256((size_t)n_pages * sizeof(int32_t)) + up256((size_t)n_seqs * sizeof(int2));
}

int page_pieces(size_t bytes) { return (int)((bytes + kMoveBytes - 1) / kMoveBytes); }

cudaError_t launch_pages_extend(const PagePool& p, const PageList& l, int steps, const int32_t* count, int32_t* slot,
                                void* scratch, int32_t* status, cudaStream_t stream) {
  PoolParams a = params_of(p, scratch);
  a.seq = l.seq;
  a.n = l.n;
  a.steps = steps;
  a.arg = count;
  a.slot = slot;
  a.status = status;
  return launch_plan<kExtend>(a, stream);
}

cudaError_t launch_pages_trim(const PagePool& p, const PageMoves* caches, const PageList& l, const int32_t* new_len,
                              void* scratch, int32_t* status, cudaStream_t stream) {
  PoolParams a = params_of(p, scratch);
  a.seq = l.seq;
  a.n = l.n;
  a.arg = new_len;
  a.status = status;
  const cudaError_t e = launch_plan<kTrim>(a, stream);
  if (e != cudaSuccess || caches->caches == 0) return e;
  return launch_moves<kNoRows>(a, moves_of(a, caches), (long long)l.n * caches->first[caches->caches], stream);
}

cudaError_t launch_pages_fork(const PagePool& p, const PageMoves* caches, const int32_t* src, const int32_t* dst, int n,
                              void* scratch, int32_t* status, cudaStream_t stream) {
  PoolParams a = params_of(p, scratch);
  a.seq = src;
  a.to = dst;
  a.n = n;
  a.status = status;
  const cudaError_t e = launch_plan<kFork>(a, stream);
  if (e != cudaSuccess) return e;
  const long long pieces = (long long)n * caches->first[caches->caches];
  return launch_moves<kForkRows>(a, moves_of(a, caches), pieces > n ? pieces : n, stream);
}

cudaError_t launch_pages_free(const PagePool& p, const PageList& l, void* scratch, int32_t* status, cudaStream_t stream) {
  PoolParams a = params_of(p, scratch);
  a.seq = l.seq;
  a.n = l.n;
  a.status = status;
  return launch_plan<kFree>(a, stream);
}

cudaError_t launch_pages_compact(const PagePool& p, const PageMoves* caches, int32_t* n_live, void* scratch,
                                 int32_t* status, cudaStream_t stream) {
  PoolParams a = params_of(p, scratch);
  a.n_live = n_live;
  a.status = status;
  Launch l(kCluster, kPlanThreads, 0, stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, pages_compact_kernel, a);
  if (e != cudaSuccess) return e;
  const long long pieces = (long long)(p.n_pages / 2) * caches->first[caches->caches];
  return launch_moves<kRemapRows>(a, moves_of(a, caches), pieces > p.n_seqs ? pieces : p.n_seqs, stream);
}

cudaError_t launch_pages_copy(const PageMoves& m, cudaStream_t stream) {
  MoveParams v = {};
  v.m = m;
  return launch_moves<kNoRows>(PoolParams{}, v, (long long)m.n * m.first[m.caches], stream);
}

}  // namespace gdn
