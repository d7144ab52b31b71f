// packed_search.h -- the search for a packed row's sequence (gfx950).
#pragma once

#include "fp8bs_device.h"

namespace fp8bs {

// Largest b in 0 .. B-1 with key(b) <= t, for a non-decreasing key with
// key(0) <= t: 64 probes at a time, one to a lane of the wave, so 64
// sequences cost one load, 4096 two.  Every lane of the wave must call it.
template <typename Key>
__device__ __forceinline__ int search64(int B, int64_t t, Key key) {
  const int lane = static_cast<int>(threadIdx.x) & 63;
  int lo = 0, n = B;   // the answer lies in lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 63) >> 6;
    const int p = lane * step;
    const bool le = p < n && key(lo + p) <= t;
    const int cnt = __popcll(__ballot(le));          // le holds for a prefix of the lanes
    const int first = (cnt > 0 ? cnt - 1 : 0) * step;
    lo += first;
    n = n - first < step ? n - first : step;
  }
  return lo;
}

}  // namespace fp8bs
