// What the kernels over the paged K/V cache share: the batch's ragged layout
// (query_start [R + 1]), the split of its attention into query tiles and key
// tiles, and the search from a grid unit to its request.
#pragma once
#include <cstdint>
#include <algorithm>
#include <mutex>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "sm103_ptx.cuh"
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
  __device__ __forceinline__ int window_lo(const PagedAttnArgs& a, int t) const {
    return a.window > 0 ? (int)max((int64_t)pos(t) - a.window + 1, (int64_t)0) : 0;
  }
  __device__ __forceinline__ int lo(const PagedAttnArgs& a, int t) const {
    const int x = window_lo(a, t);
    return a.doc_start ? max(x, __ldg(a.doc_start + t)) : x;
  }
};

// Key tiles [first, first + count) of a query tile; one (of no visible key) where nothing is seen.
__device__ __forceinline__ void key_tiles(int lo, int hi, int& first, int& count) {
  first = hi > lo ? lo / kKeyTile : 0;
  count = hi > lo ? (hi + kKeyTile - 1) / kKeyTile - first : 1;
}

// The sequence of key tiles of a call: requests, their query tiles (tq tokens
// each), the K/V heads, the key tiles, each unit's (query tile's and head's)
// behind unit_cost places that stand for its start and end.  `ctas` CTAs take
// equal contiguous ranges of it, so a unit's keys may be split over consecutive
// CTAs: each then leaves a partial result, and the first of them a record for
// the merge.
__device__ __forceinline__ int64_t range_begin(int64_t c, int64_t total, int ctas) { return c * total / ctas; }
// The CTA whose range holds tile x.
__device__ __forceinline__ int range_of(int64_t x, int64_t total, int ctas) {
  return (int)(((x + 1) * ctas - 1) / total);
}

// One CTA's share of one (query tile, K/V head).
struct Segment {
  int n;               // key tiles; 0: the CTA's range has ended
  int kt;              // the first of them (they are taken from the last down)
  int r, g;            // request, K/V head
  int h0, heads;       // query heads
  int t0, ntok;        // rows
  int lo, hi;          // keys that some row sees
  int all_lo, all_hi;  // keys that every row sees
  int slot;            // partial result to write: 0 (begun by an earlier CTA), 1 (begun here), -1: the whole unit
};

// A split unit, at the CTA that began it; its partial results are that CTA's
// slot 1 and the following parts - 1 CTAs' slot 0 (CTA c: slots 2 c, 2 c + 1).
struct PagedMerge {
  int t0, ntok, h0, heads, parts;  // parts = 0: no unit begun by this CTA is split
};

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kTop = 8.75f;      // P = 2^(x - m') <= 2^8.75 < 431 (e4m3: 448)
constexpr float kRefresh = 4.25f;  // a refreshed m' puts the tile's maximum at 2^4.25
constexpr float kNoMax = -3e38f;   // m' of a row that has seen nothing

__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N, uint32_t a_mn, uint32_t b_mn) {
  return (1u << 4) | (a_mn << 15) | (b_mn << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// True in every thread if it is in any of the `n` threads at the named barrier.
__device__ __forceinline__ bool bar_any(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float warp_max(float x) {  // NaN only if all are
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// Float arithmetic two at a time.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Offset of 16-byte chunk ch of row r, rows of D bytes under the D-byte swizzle.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int ch) {
  return (uint32_t)(r * D + ((D == 128 ? ch ^ (r & 7) : ch ^ ((r >> 1) & 3)) << 4));
}

// tanh(u) / u as a polynomial of u^2 <= 0.5: the one of degree 4 through the Chebyshev
// points of [0, 0.5], to within 4 x 2^-23 of the value.  Caps are wide as a rule, so
// that most keys need no exponential and no reciprocal for theirs (prompts of packed
// documents: 94 us when this came, without it 100).
constexpr float kTanhTop = 0.5f;  // of u^2
__device__ constexpr float kTanh[5] = {0.99999964f, -0.33329946f, 0.13277967f, -0.05072029f, 0.01364212f};
// tanh(u) for any u, to within 8 x 2^-23 of the value: the polynomial where it holds, else
// 1 - 2 / (1 + e^(2 u)), which is good to a few 2^-23 of 1 only.
__device__ __forceinline__ float tanh_any(float u) {
  const float u2 = u * u;
  float y = kTanh[4];
#pragma unroll
  for (int d = 3; d >= 0; --d) y = fmaf(y, u2, kTanh[d]);
  const float far = fmaf(-2.f, __fdividef(1.f, 1.f + ex2_approx(u * (2.f * kLog2e))), 1.f);
  return u2 <= kTanhTop ? u * y : far;
}

// 8 bf16 values of a row whose largest magnitude has the bits amax, in two
// e4m3 terms of q 2^s: s puts amax = (1 + f) 2^e to at most 448 = 1.75 * 2^8.
// back = 2^-s, NaN for a row with an infinity or NaN: it has no finite result.
__device__ __forceinline__ void split_q8(const uint32_t (&w)[4], uint32_t amax, uint32_t (&hi)[2], uint32_t (&lo)[2],
                                         float& back) {
  int s = 8 - ((int)(amax >> 23) - 127) - ((amax & 0x7fffffu) > 0x600000u);
  s = amax == 0u ? 0 : min(s, 120);
  const float f = __uint_as_float((uint32_t)(s + 127) << 23);
  back = amax >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 - s) << 23);
  hi[0] = hi[1] = lo[0] = lo[1] = 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float y0 = __uint_as_float(w[k] << 16) * f, y1 = __uint_as_float(w[k] & 0xffff0000u) * f;
    const uint32_t c = e4m3x2(y0, y1);
    const float2 d = e4m3x2_f32(c);
    hi[k >> 1] |= c << (16 * (k & 1));
    lo[k >> 1] |= e4m3x2(y0 - d.x, y1 - d.y) << (16 * (k & 1));
  }
}

// Set when a wait of any call on the device runs out, whichever workspace the call had: one that is
// allocated for a call is gone when its caller asks.  One word per file that includes this.
__device__ int g_timed_out;

// mbar_wait with its slow part out of line, so that the roles' loops stay
// small, with a long suspension per probe, so that waiting warps leave the
// issue slots to the others, and without a look at the (slow) clock before a
// few probes have run out: the same time limit and abort flag.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* cta_abort, int* status) {
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(100000u)
        : "memory");
    if (ok) return true;
    if (*cta_abort) return false;
    if (i < 16) continue;
    if (i == 16) t0 = globaltimer_ns();
    else if (globaltimer_ns() - t0 > kWaitLimitNs) break;
  }
  *cta_abort = 1;
  atomicExch(status, kDevWaitTimeout);  // (whatever an uninitialised workspace held)
  atomicExch(&g_timed_out, kDevWaitTimeout);
  return false;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* cta_abort, int* status) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, cta_abort, status);
}

// One thread that waits for what never comes, and so reports a wait that ran out.
__global__ void paged_wait_check_kernel(int* status) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  abort_flag = 0;
  mbar_init(&bar, 1);
  mbar_fence_init();
  wait_bar(&bar, 0, &abort_flag, status);
}
cudaError_t wait_check(int* status, cudaStream_t stream) {
  paged_wait_check_kernel<<<1, 1, 0, stream>>>(status);
  return cudaGetLastError();
}
cudaError_t timed_out_word(int** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_timed_out); }

// Place in a ring of N slots with a barrier each: index and the parity of its
// phase (no divisions in the roles' loops).
template <int N>
struct Ring {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      phase ^= 1u;
    }
  }
};

struct PagedParams {
  PagedAttnArgs a;
  // Rows of a query tile: tq tokens x up to Gr of the G heads of a K/V head; more than C heads are cut into
  // `cuts` groups, which the sequence of units counts as K/V heads of their own (HV = HK * cuts).
  int G, Gr, cuts, HV, tq;
  int ctas;
  int unit_cost;        // what a segment costs beyond its tiles, in tiles
  int* status;
  PagedMerge* merge;    // [ctas]
  float* part_ml;       // [2 ctas][m' | l][C]
  float* part_o;        // [2 ctas][C][D]
  float* q_scale;       // [T, H], of a q split beforehand
  const int32_t* tile_doc;  // first document start of each query tile, if found beforehand (see tile_slot)
};

// Query tile (ta - t0) / tq of request r among those of the batch, with room
// for every request's: request r's begin at floor(t0 / tq) + r.
__device__ __forceinline__ int tile_slot(const PagedParams& p, int r, int t0, int ta) {
  return t0 / p.tq + r + (ta - t0) / p.tq;
}
// Keys [lo, hi) that hold all that rows ta .. tb - 1 see.
__device__ __forceinline__ void tile_range(const PagedParams& p, const PagedRequest& q, int r, int ta, int tb, int& lo,
                                           int& hi) {
  lo = q.window_lo(p.a, ta);
  hi = q.hi(tb - 1);
  if (p.a.doc_start) {
    int doc = 0x7fffffff;
    if (p.tile_doc)
      doc = p.tile_doc[tile_slot(p, r, q.t0, ta)];
    else
      for (int t = ta; t < tb; ++t) doc = min(doc, __ldg(p.a.doc_start + t));
    lo = max(lo, doc);
  }
}

// Places of a unit of request r whose first row is t.
__device__ __forceinline__ int unit_places(const PagedParams& p, const PagedRequest& q, int r, int t) {
  int lo, hi, first, count;
  tile_range(p, q, r, t, min(t + p.tq, q.t1), lo, hi);
  key_tiles(lo, hi, first, count);
  return count + p.unit_cost;
}
// Places of request r in the sequence (over its query tiles begin, begin + step, ... and the K/V heads).
__device__ __forceinline__ int64_t request_places(const PagedParams& p, int r, int begin, int step) {
  PagedRequest q;
  q.load(p.a, r);
  int64_t n = 0;
  for (int64_t t = q.t0 + (int64_t)begin * p.tq; t < q.t1; t += (int64_t)step * p.tq) n += unit_places(p, q, r, (int)t);
  return n * p.HV;
}

// Exclusive prefix sums of v[0 .. R-1] in place, the total in v[R]; all
// threads.  v has room for a word per warp behind that.
template <int kThreads>
__device__ void scan_tiles(int64_t* v, int R) {
  int64_t* warp_sum = v + R + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (R + kThreads - 1) / kThreads;
  const int beg = min(tid * per, R), end = min(beg + per, R);
  int64_t sum = 0;
  for (int i = beg; i < end; ++i) sum += v[i];
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(kAll, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int64_t run = inc - sum;
  for (int w = 0; w < warp; ++w) run += warp_sum[w];
  for (int i = beg; i < end; ++i) {
    const int64_t x = v[i];
    v[i] = run;
    run += x;
  }
  if (tid == kThreads - 1) v[R] = run;
  __syncthreads();
}

// This CTA's range of the sequence, and where it begins.
struct PagedRange {
  int64_t x0, x1, total, off0;  // off0: tiles of request r0 before x0
  int ctas, r0;
};

__device__ __forceinline__ void set_range(PagedRange& g, const PagedParams& p, int64_t total) {
  g.total = total;
  // with fewer tiles than CTAs the first CTAs take one each: a unit's parts are consecutive CTAs
  g.ctas = (int)min((int64_t)p.ctas, total);
  if ((int)blockIdx.x < g.ctas) {
    g.x0 = range_begin(blockIdx.x, total, g.ctas);
    g.x1 = range_begin((int64_t)blockIdx.x + 1, total, g.ctas);
  }
}

// By all threads of the CTA; `prefix`: shared memory for R + 1 words and one per warp.  Valid in warp `walker` only.
template <int kThreads>
__device__ __forceinline__ PagedRange paged_range(const PagedParams& p, int64_t* prefix, int walker) {
  const int R = p.a.R, lane = threadIdx.x & 31;
  const bool walks = (int)threadIdx.x >> 5 == walker;
  PagedRange g{};
  // A small call, few query tiles: in that warp's registers, without the others and the barriers between (one
  // request of 1000 tokens: 11.3 us by all threads, 10.6 so; five prompts of 3250 tokens: 76 and 79).
  if (R <= 32 && p.a.T / p.tq + R <= 64) {
    if (!walks) return g;
    int per = 32;
    while (per * R > 32) per >>= 1;
    const int r = lane / per, sub = lane & (per - 1);
    int64_t n = r < R ? request_places(p, r, sub, per) : 0;
    for (int o = 1; o < per; o <<= 1) n += __shfl_xor_sync(kAll, n, o);
    if (sub != 0) n = 0;
    int64_t inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(kAll, inc, o);
      if (lane >= o) inc += u;
    }
    set_range(g, p, __shfl_sync(kAll, inc, 31));
    // the last request that begins at or before x0
    const int at = 31 - __clz((int)__ballot_sync(kAll, sub == 0 && r < R && inc - n <= g.x0));
    g.r0 = at / per;
    g.off0 = g.x0 - __shfl_sync(kAll, inc - n, at);
    return g;
  }
  // as many lanes a request as there are threads for
  int per = 1;
  while (per < 32 && 2 * per * R <= kThreads) per *= 2;
  if (per == 1) {
    for (int r = threadIdx.x; r < R; r += kThreads) prefix[r] = request_places(p, r, 0, 1);
  } else {
    const int r = threadIdx.x / per, sub = threadIdx.x & (per - 1);
    int64_t n = r < R ? request_places(p, r, sub, per) : 0;
    for (int o = 1; o < per; o <<= 1) n += __shfl_xor_sync(kAll, n, o);
    if (r < R && sub == 0) prefix[r] = n;
  }
  __syncthreads();
  scan_tiles<kThreads>(prefix, R);
  if (walks) {
    set_range(g, p, prefix[R]);
    int hi = R;
    while (hi - g.r0 > 1) {
      const int mid = (g.r0 + hi) >> 1;
      if (prefix[mid] <= g.x0) g.r0 = mid;
      else hi = mid;
    }
    g.off0 = g.x0 - prefix[g.r0];
  }
  return g;
}

// Walks the range by one warp: emit(segment, its request) for each segment in turn, until
// it returns false.  Returns the record for the merge.
template <typename F>
__device__ __forceinline__ PagedMerge walk_segments(const PagedParams& p, const PagedRange& w, F emit) {
  const PagedAttnArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  PagedMerge mine{0, 0, 0, 0, 0};
  int64_t x = w.x0, off = w.off0;
  for (int r = w.r0; x < w.x1 && r < a.R; ++r) {
    PagedRequest q;
    q.load(a, r);
    // the query tile in which the range begins, 32 tiles at a time
    int ta = q.t0;
    while (off > 0 && ta < q.t1 - p.tq) {
      const int64_t t = ta + (int64_t)lane * p.tq;
      const int n = t < q.t1 ? unit_places(p, q, r, (int)t) : 0;
      int64_t inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t before = __shfl_up_sync(kAll, inc, o);
        if (lane >= o) inc += before;
      }
      const uint32_t reach = __ballot_sync(kAll, off < inc * p.HV);
      const int k = reach ? __ffs((int)reach) - 1 : 31;
      const int64_t upto = __shfl_sync(kAll, reach ? inc - n : inc, k);
      off -= upto * p.HV;
      ta = (int)min(ta + (int64_t)(reach ? k : 32) * p.tq, (int64_t)q.t1);
      if (reach) break;
    }
    for (; ta < q.t1 && x < w.x1; ta += p.tq) {
      const int tb = min(ta + p.tq, q.t1);
      Segment s;
      tile_range(p, q, r, ta, tb, s.lo, s.hi);
      int first, count;
      key_tiles(s.lo, s.hi, first, count);
      const int len = count + p.unit_cost;  // places of a unit
      s.all_lo = q.window_lo(a, tb - 1);
      s.all_hi = q.hi(ta);
      if (a.doc_start) {
        int least = 0x7fffffff, most = 0;
        for (int t = ta + lane; t < tb; t += 32) {
          const int y = max(0, q.lo(a, t));
          least = min(least, y);
          most = max(most, y);
        }
        s.lo = __reduce_min_sync(kAll, least);
        s.all_lo = __reduce_max_sync(kAll, most);
      }
      if (s.hi <= s.lo) s.lo = s.hi = 0;  // nothing is seen: no block is read
      s.r = r;
      s.t0 = ta;
      s.ntok = tb - ta;
      for (int v = (int)(off / len); v < p.HV && x < w.x1; ++v) {
        const int skip = (int)(off - (int64_t)v * len);  // places of this unit before this CTA's range
        off = (int64_t)(v + 1) * len;
        const int take = (int)min((int64_t)(len - skip), w.x1 - x);
        const int64_t last = x + (len - skip) - 1;  // the unit's last place
        x += take;
        const int beg = max(0, skip - p.unit_cost), end = max(0, skip + take - p.unit_cost);  // tiles
        if (beg == end) continue;
        s.g = v / p.cuts;
        s.h0 = s.g * p.G + v % p.cuts * p.Gr;
        s.heads = min(p.Gr, p.G - v % p.cuts * p.Gr);
        s.kt = first + beg;
        s.n = end - beg;
        s.slot = beg == 0 ? (end == count ? -1 : 1) : 0;
        if (s.slot == 1)
          mine = PagedMerge{ta, s.ntok, s.h0, s.heads, range_of(last, w.total, w.ctas) - (int)blockIdx.x + 1};
        const int gone = min(s.lo / kKeyTile - s.kt, s.n - 1);  // one tile stays: the result is due
        if (gone > 0) {
          s.kt += gone;
          s.n -= gone;
        }
        if (!emit(s, q)) return mine;
      }
      off = 0;
    }
  }
  return mine;
}

// The units that several CTAs share: out = sum_i w_i O_i / sum_i w_i l_i, w_i =
// 2^(m_i - max m), lse = max m + log2 of the latter sum.  blockIdx.x: the CTA that
// began the unit.  D / 32 value columns a lane, kWarps warps a row, whose sums meet
// in shared memory.  Bound by latency: two dependent reads, with the parts' values
// in flight together.  8 us behind 64 requests' decode, 17 us behind three prompts of up to
// 2500 tokens (19 MB of parts).
constexpr int kMaxParts = 1024;
template <int C>
constexpr int kMergeThreads = C == 256 ? 256 : 128;  // (a prompt of 300 tokens: 23.2 us with 256, 24.4 with 128)

template <int D, int C, int kWarps>
__global__ void __launch_bounds__(kMergeThreads<C>) paged_merge_kernel(const __grid_constant__ PagedParams p) {
  constexpr int kPer = D / 32;
  __shared__ float warp_acc[kWarps][D], warp_sum[kWarps];
  grid_dependency_wait();
  const PagedMerge u = p.merge[blockIdx.x];
  const int lane = threadIdx.x & 31, warp = (int)threadIdx.x >> 5, share = warp % kWarps;
  const int c = (int)blockIdx.y * (kMergeThreads<C> / 32 / kWarps) + warp / kWarps;
  if (c >= u.ntok * u.heads || u.parts == 0) return;  // (the same for the warps of a row)
  // the parts: slot 1 of this CTA, then slot 0 of the following ones
  const int64_t first = 2 * (int64_t)blockIdx.x;
  auto part = [&](int i) { return first + (i == 0 ? 1 : 2 * i); };
  float top = kNoMax;
  for (int i = lane; i < u.parts; i += 32) top = fmaxf(top, p.part_ml[part(i) * 2 * C + c]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  float sum = 0.f, acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  for (int base = share; base < u.parts; base += 32 * kWarps) {  // this warp's: base, base + kWarps, ...
    float w = 0.f;
    if (base + kWarps * lane < u.parts) {
      const float* ml = p.part_ml + part(base + kWarps * lane) * 2 * C + c;
      w = ex2_approx(ml[0] - top);
      sum = fmaf(w, ml[C], sum);
    }
    const int n = min(32, (u.parts - base + kWarps - 1) / kWarps);
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const float f = __shfl_sync(kAll, w, j);
      const float* o = p.part_o + (part(base + kWarps * j) * C + c) * D + kPer * lane;
      if (kPer == 4) {
        const float4 v = *reinterpret_cast<const float4*>(o);
        acc[0] = fmaf(f, v.x, acc[0]);
        acc[1] = fmaf(f, v.y, acc[1]);
        acc[kPer - 2] = fmaf(f, v.z, acc[kPer - 2]);
        acc[kPer - 1] = fmaf(f, v.w, acc[kPer - 1]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(o);
        acc[0] = fmaf(f, v.x, acc[0]);
        acc[1] = fmaf(f, v.y, acc[1]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  if (kWarps > 1) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) warp_acc[share][kPer * lane + k] = acc[k];
    if (lane == 0) warp_sum[share] = sum;
    __syncthreads();
    if (share > 0) return;
#pragma unroll
    for (int i = 1; i < kWarps; ++i) {
      sum += warp_sum[i];
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] += warp_acc[i][kPer * lane + k];
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t row = (int64_t)(u.t0 + c / u.heads) * p.a.H + u.h0 + c % u.heads;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.a.out) + row * D + kPer * lane);
#pragma unroll
  for (int k = 0; k < kPer / 2; ++k) dst[k] = pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
  if (lane == 0) p.a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// A cache as rows of D bytes, a box one block of one head, the D-byte swizzle;
// rows behind the cache read as zeros.
cudaError_t cache_map(CUtensorMap* m, const void* cache, int64_t rows, int D) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)D};
  const cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)kBlock}, es[2] = {1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(cache), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// The call's workspace: status word, merge records, partial m' and l, partial O.
struct PagedSizes {
  int ctas;
  size_t merge, ml, o, bytes;
};
inline PagedSizes paged_sizes(int C, int D, int per_sm, int num_sms) {
  PagedSizes s;
  s.ctas = std::min(num_sms * per_sm, kMaxParts);
  s.merge = kWsStatusBytes;
  s.ml = s.merge + align256(sizeof(PagedMerge) * s.ctas);
  s.o = s.ml + align256((size_t)2 * s.ctas * 2 * C * 4);
  s.bytes = s.o + (size_t)2 * s.ctas * C * D * 4;
  return s;
}

// The parameters of a call with C rows per query tile, without those of a
// split q; per_sm CTAs an SM.
template <int C>
PagedParams paged_params(const PagedAttnArgs& a, const PagedSizes& sz, int unit_cost) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  PagedParams p{};
  p.a = a;
  p.G = a.H / a.HK;
  p.cuts = (p.G + C - 1) / C;
  p.Gr = (p.G + p.cuts - 1) / p.cuts;
  p.HV = a.HK * p.cuts;
  // 256 rows are two halves of whole tokens
  p.tq = C == 256 ? 2 * (128 / p.Gr) : std::max(1, C / p.Gr);
  p.ctas = sz.ctas;
  p.unit_cost = unit_cost;
  p.status = reinterpret_cast<int*>(ws);
  p.merge = reinterpret_cast<PagedMerge*>(ws + sz.merge);
  p.part_ml = reinterpret_cast<float*>(ws + sz.ml);
  p.part_o = reinterpret_cast<float*>(ws + sz.o);
  return p;
}

// A launch that may overlap the preceding kernel's end (the kernels wait for it
// before they touch global memory).
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream,
                              const Args&... args) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int C, int kWarps>
cudaError_t launch_merge_warps(const PagedParams& p, cudaStream_t stream) {
  return launch_overlapped(paged_merge_kernel<D, C, kWarps>,
                           dim3((unsigned)p.ctas, (unsigned)(C * kWarps / (kMergeThreads<C> / 32))), kMergeThreads<C>, 0,
                           stream, p);
}
// Four warps a row where a unit may have 16 parts or more (few units, long tables): one request of up to 8000 tokens
// 14.8 us, 19.2 with one warp; of 1000 tokens 11.3 and 10.6; 64 of up to 16 000 177.7 and 176.0.
template <int D, int C>
cudaError_t launch_merge(const PagedParams& p, cudaStream_t stream) {
  const int64_t tiles = std::max<int64_t>(((int64_t)p.a.T + p.tq - 1) / p.tq, std::min(p.a.R, p.a.T));
  const int64_t parts = std::min<int64_t>(p.ctas / (tiles * p.HV), p.a.MB / 2 + 1);
  if (C <= 16 && parts >= 16) return launch_merge_warps<D, C, C <= 16 ? 4 : 1>(p, stream);
  return launch_merge_warps<D, C, 1>(p, stream);
}

cudaError_t cache_maps(const PagedAttnArgs& a, CUtensorMap* k_map, CUtensorMap* v_map) {
  const int64_t rows = a.NB * a.HK * kBlock;
  const cudaError_t e = cache_map(k_map, a.k_cache, rows, a.D);
  return e == cudaSuccess ? cache_map(v_map, a.v_cache, rows, a.D) : e;
}

}  // namespace

}  // namespace smla
