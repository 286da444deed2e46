// warp_search.cuh -- a 32-way search by a whole warp.
#pragma once

namespace pa {
namespace {

// The largest i in [0, n) that pred holds for, where pred holds for 0 (it is
// not asked) and then for a first part of the indexes: one round of probes up
// to n = 32, two up to 1024.  Where pred is not of that kind some index in [0, n)
// comes back.
template <typename Pred>
__device__ __forceinline__ int warp_search_last(int n, int lane, Pred pred) {
  int lo = 0;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int stride = (n - 1) / 32 + 1;
    const bool holds = lane == 0 || (static_cast<long long>(lane) * stride < n && pred(lo + lane * stride));
    const int last = __popc(__ballot_sync(0xffffffffu, holds)) - 1;
    n = min(stride, n - last * stride);
    lo += last * stride;
  }
  return lo;
}

}  // namespace
}  // namespace pa
