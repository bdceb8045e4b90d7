// gdn_attn_ranges.h -- which of a job's ranges the join of gdn_attn_decode_shared
// reads.  Plain C++, so that it is tested without a GPU.
#pragma once

#ifdef __CUDACC__
#define GDN_ANYWHERE __host__ __device__ __forceinline__
#else
#define GDN_ANYWHERE inline
#endif

namespace gdn {

struct Ranges {
  int first, count;   // shares [first, first + count)
};

// The shares from `first` to `last`, as the first kernel noted them for a job.  Where
// one of its waits gave up it noted nothing, and the words hold whatever the caller's
// workspace did: whatever they are, what comes back lies in [0, shares).
GDN_ANYWHERE Ranges ranges_of(int first, int last, int shares) {
  if (first < 0 || first >= shares || last < first) return Ranges{0, 0};
  if (last >= shares) last = shares - 1;
  return Ranges{first, last - first + 1};
}

}  // namespace gdn
