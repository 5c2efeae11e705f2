// What the kernels over the paged K/V cache share: the batch's ragged layout
// (query_start [R + 1]), the split of its attention into query tiles and key
// tiles, and the search from a grid unit to its request.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "smla_common.cuh"
#include "smla_kernels.h"

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

constexpr int kKeyTile = 128;  // keys per tile: two blocks of the cache

// A request of the batch as the attention sees it.
struct PagedRequest {
  int t0, t1;  // its rows
  int len;     // its tokens
  int kmax;    // keys that its table row can hold
  int prefix;

  __device__ __forceinline__ void load(const PagedAttnArgs& a, int r) {
    t0 = clamp_start(a.query_start, r, a.T);
    t1 = max(t0, clamp_start(a.query_start, r + 1, a.T));
    len = max(0, __ldg(a.seq_lens + r));
    kmax = (int)min((int64_t)len, (int64_t)a.MB * kBlock);
    prefix = a.prefix_lens ? __ldg(a.prefix_lens + r) : 0;
  }
  __device__ __forceinline__ int pos(int t) const { return len - t1 + t; }
  // visible keys [lo, hi) of row t
  __device__ __forceinline__ int hi(int t) const { return min(kmax, max(pos(t) + 1, prefix)); }
  __device__ __forceinline__ int lo(const PagedAttnArgs& a, int t) const {
    int x = a.window > 0 ? max(0, (int)max((int64_t)pos(t) - a.window + 1, (int64_t)0)) : 0;
    return a.doc_start ? max(x, __ldg(a.doc_start + t)) : x;
  }
  // Union [lo, hi) of the rows ta .. tb - 1's visible keys, and the keys
  // [all_lo, all_hi) that all of them see.
  __device__ __forceinline__ void range(const PagedAttnArgs& a, int ta, int tb, int& lo_, int& hi_, int& all_lo,
                                        int& all_hi) const {
    hi_ = hi(tb - 1);
    all_hi = hi(ta);
    lo_ = lo(a, ta);
    all_lo = lo(a, tb - 1);
    if (a.doc_start)
      for (int t = ta; t < tb; ++t) {
        const int x = lo(a, t);
        lo_ = min(lo_, x);
        all_lo = max(all_lo, x);
      }
  }
};

// Key tiles [first, first + count) of a query tile; one (of no visible key) where nothing is seen.
__device__ __forceinline__ void key_tiles(int lo, int hi, int& first, int& count) {
  first = hi > lo ? lo / kKeyTile : 0;
  count = hi > lo ? (hi + kKeyTile - 1) / kKeyTile - first : 1;
}

// The sequence of key tiles of a call: requests, their query tiles (tq tokens
// each), the K/V heads, the key tiles.  `ctas` CTAs take equal contiguous
// ranges of it, so a query tile's keys may be split over consecutive CTAs:
// each then leaves a partial result, and the first of them a record for the
// merge.
__device__ __forceinline__ int64_t range_begin(int64_t c, int64_t total, int ctas) { return c * total / ctas; }
// The CTA whose range holds tile x.
__device__ __forceinline__ int range_of(int64_t x, int64_t total, int ctas) {
  return (int)(((x + 1) * ctas - 1) / total);
}

// One CTA's share of one (query tile, K/V head).
struct Segment {
  int r, g;          // request, K/V head
  int h0, heads;     // query heads
  int t0, ntok;      // rows
  int pos0;          // position of row t0
  int kt, n;         // key tiles kt .. kt + n - 1
  int lo, hi;        // keys that some row sees
  int all_lo, all_hi;  // keys that every row sees
  int slot;          // partial result to write: 0 (begun by an earlier CTA), 1 (begun here), -1: the whole unit
  int parts;         // slot 1: CTAs that share the unit
};

// A partial result's place: CTA c's slots 2 c and 2 c + 1.
struct PagedMerge {
  int t0, ntok, h0, heads, parts;  // parts = 0: no unit begun by this CTA is split
};

}  // namespace smla
