// What the kernels over the paged K/V cache share: the batch's ragged layout
// (query_start [R + 1]) and the search from a grid unit to its request.
#pragma once
#include <cstdint>

namespace smla {

// query_start[i] inside [0, T]: whatever it holds, no token index leaves the batch.
__device__ __forceinline__ int clamp_start(const int32_t* __restrict__ query_start, int i, int T) {
  return max(0, min(__ldg(query_start + i), T));
}

// The last r in [0, R) with first(r) <= u, first non-decreasing with first(0)
// <= u; by all lanes of a warp together, 32 probes a round (one memory round
// trip up to 32 requests, two up to 1024).
template <typename F>
__device__ __forceinline__ int search_units(int R, int u, F first) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = R;  // the answer lies in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int i = lo + lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, i < hi && (lane == 0 || first(i) <= u));
    const int k = 31 - __clz((int)le);
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

}  // namespace smla
