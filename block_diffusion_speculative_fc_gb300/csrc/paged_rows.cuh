// The request that owns a row of a ragged batch.
#pragma once
#include "common.cuh"
#include "target_ops.h"

namespace dflash {

struct RowOwner {
  int b, start, kv;   // request, its first row, its kv_len
};

// Called by every thread of a CTA: the request whose range holds row t, or false
// (no owner, or two: flagged).  Ranges that are none are flagged by row 0's CTA.
// kv_len is read beside row_start, not after it: one load's latency less.
__device__ __forceinline__ bool owner_of_row(const PagedRows &r, int t, unsigned int *err,
                                             RowOwner *s_owner) {
  int found = 0;
  for (int i = threadIdx.x; i < r.B; i += blockDim.x) {
    const int a = r.row_start[i], e = r.row_start[i + 1], kv = r.kv_len[i];
    const bool range = a >= 0 && a <= e && e <= r.total_rows;
    if (!range && t == 0) raise_error(err, DFLASH_DERR_ROW_RANGE);
    if (range && a <= t && t < e) {
      ++found;
      *s_owner = {i, a, kv};
    }
  }
  const bool twice = __syncthreads_or(found > 1) != 0;
  const int owners = __syncthreads_count(found);
  if (owners == 1 && !twice) return true;
  if (owners > 0 && threadIdx.x == 0) raise_error(err, DFLASH_DERR_ROW_RANGE);
  return false;
}

}  // namespace dflash
