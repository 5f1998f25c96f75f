// Where a ragged row lives in a paged cache: plain integer arithmetic, shared by the kernels and the host.
#pragma once

#include "ops.h"

#ifdef __HIPCC__
#define MX_HD __host__ __device__ inline
#else
#define MX_HD inline
#endif

// The cache slot of row t: -1 where the position has none, -2 where the row belongs to no sequence.
MX_HD int64_t slot_of(const CacheArgs& a, int64_t t) {
  // sequences that end at or before t
  int lo = 0, hi = a.n_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)a.cu[mid + 1] <= t) lo = mid + 1; else hi = mid;
  }
  if (lo >= a.n_seqs || t < (int64_t)a.cu[lo]) return -2;
  const int64_t pos = t - a.cu[lo] + (a.start ? a.start[lo] : 0);
  if (pos < 0) return -1;
  const int64_t p = pos / a.page_size;
  if (p >= a.max_pages) return -1;
  const int64_t page = a.table[(int64_t)lo * a.ld_table + p];
  if (page < 0 || page >= a.num_pages) return -1;
  return page * a.page_size + (pos - p * a.page_size);
}
