// Quantize-and-store of new K and V rows into the paged 8-bit K/V cache: e4m3
// codes [NB, HK, 64, D] with one scale per block of 64 tokens and head.
//
// A block's scale is a power of two 2^E, E the smallest (from -100 up) with
// amax <= 448 * 2^E over the rows it covers, so dividing by it is exact and the
// only rounding is that to e4m3.  A block whose first row is written by this
// call takes the new rows' scale.  A block partly filled before keeps the
// larger of its own and the new rows' scale; where that grows, the codes of
// its old rows become e4m3(code * old / new), exact but for codes that turn
// subnormal.  A block that another program has begun may have any scale: it
// goes a way of its own, in which quotients and products are rounded once too.  Infinities saturate and are left out of amax; NaN is stored as
// 0, so that no stored row can spread NaN to a query that does not see it.
//
// The new rows of a block are found from the batch's lengths (the tokens of a
// request are consecutive), not from a slot map: the block's scale needs them
// together, and this way one warp has them without any exchange or atomics.
// Unit u of the grid stands for one touched block: request r's units start at
// floor(query_start_r / 64) + 2 r, which leaves room for every block that its
// tokens can touch, so a unit finds its request by a search in query_start.
// One warp or four per (block, head, K or V); the new rows are read once, so the
// kernel moves what it must: bound by HBM for prefill, by latency for single
// tokens.  Measured at 8 heads, D = 128, replayed from a graph: 9 requests of up to
// 3500 tokens (148 MB) 25.8 us, 5.7 TB/s, 0.84 of the copy bandwidth; 64 single tokens 2.9 us.
#include "smla_paged.cuh"

namespace smla {

namespace {

constexpr int kStoreWarps = 8;

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// |bf16| of both halves of w, 0 for infinities and NaN, into amax.
__device__ __forceinline__ float finite_amax(float amax, uint32_t w) {
  const float lo = fabsf(__uint_as_float(w << 16)), hi = fabsf(__uint_as_float(w & 0xffff0000u));
  if (lo < INFINITY) amax = fmaxf(amax, lo);
  if (hi < INFINITY) amax = fmaxf(amax, hi);
  return amax;
}
// Both halves of w, NaN as 0.
__device__ __forceinline__ uint32_t nan_to_0(uint32_t w) {
  if ((w & 0x7fffu) > 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7fff0000u) > 0x7f800000u) w &= 0xffffu;
  return w;
}

// Exponent E of the scale of a group with this amax (finite, >= 0): amax =
// (1 + f) 2^e, and 448 = 1.75 * 2^8.  Subnormal bf16 have e = -127 here, far
// below the floor of -100.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  return max(-100, (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The scale of a block and head, and 1 / scale: `old` is its scale before (0
// where no earlier row counts), amax its new rows'.
__device__ __forceinline__ void block_scale(float old, uint32_t amax, float& s, float& inv) {
  const int e = scale_exponent(__uint_as_float(amax));
  s = pow2(e);
  inv = pow2(-e);
  if (old > s) {
    s = old;
    inv = __frcp_rn(old);
  }
}

// Codes of the earlier rows (words of them, by `threads` threads) under a
// scale that has grown from old = f * the new one.
__device__ __forceinline__ void rescale_codes(uint32_t* __restrict__ w, int words, float f, int thread, int threads) {
#pragma unroll 8
  for (int i = thread; i < words; i += threads) {
    const uint32_t c = w[i];
    const float2 a = e4m3x2_f32(c & 0xffffu), b = e4m3x2_f32(c >> 16);
    w[i] = e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
  }
}

__device__ __forceinline__ uint32_t codes_of(uint2 v, float inv) {
  return e4m3x4(__uint_as_float(v.x << 16) * inv, __uint_as_float(v.x & 0xffff0000u) * inv,
                __uint_as_float(v.y << 16) * inv, __uint_as_float(v.y & 0xffff0000u) * inv);
}

// x, where `r` tells on which side of it the exact value lies that it was rounded from: that value rounded to the
// odd one of the float32 beside it, from which a further rounding to fewer bits goes as from the value itself.
__device__ __forceinline__ float to_odd(float x, float r) {
  if (r == 0.f || !(fabsf(x) > 0x1p-30f && fabsf(x) < INFINITY)) return x;
  const uint32_t b = __float_as_uint(x);
  return __uint_as_float(((r < 0.f) != (x < 0.f) ? b - 1u : b) | 1u);
}
__device__ __forceinline__ float product(float x, float f) {
  const float p = x * f;
  return to_odd(p, fmaf(x, f, -p));
}
__device__ __forceinline__ float quotient(float x, float m) {
  const float q = __fdiv_rn(x, m);
  return q == q ? to_odd(q, fmaf(-q, m, x)) : 0.f;  // (NaN: infinity under an infinite scale)
}

// store_rows (below) in a block whose scale is no power of two, out of line and as simple as that.
template <int D, int kGroup>
__device__ __noinline__ void store_rows_any(const __nv_bfloat16* src, int64_t stride, int row0, int n, uint8_t* page,
                                            float* scale, float old, int t, int bar, uint32_t* shared_max) {
  constexpr int kThreads = 32 * kGroup;
  auto at = [&](int i) { return __ldg(reinterpret_cast<const uint2*>(src + i / (D / 4) * stride + 4 * (i % (D / 4)))); };
  float most = 0.f;
  for (int i = t; i < n * (D / 4); i += kThreads) most = finite_amax(finite_amax(most, at(i).x), at(i).y);
  uint32_t top = __reduce_max_sync(kAll, __float_as_uint(most));
  if (kGroup == 4) {
    if ((t & 31) == 0) shared_max[t >> 5] = top;
    named_bar_sync(bar, 128);  // and every warp has read the old scale
    top = max(max(shared_max[0], shared_max[1]), max(shared_max[2], shared_max[3]));
  }
  const float need = pow2(scale_exponent(__uint_as_float(top)));
  const float s = fmaxf(old, need);
  if (old < s) {
    const float f = old * pow2(-scale_exponent(__uint_as_float(top)));
    uint32_t* w = reinterpret_cast<uint32_t*>(page);
    for (int i = t; i < row0 * (D / 4); i += kThreads) {
      const uint32_t c = w[i];
      const float2 a = e4m3x2_f32(c & 0xffffu), b = e4m3x2_f32(c >> 16);
      w[i] = e4m3x4(product(a.x, f), product(a.y, f), product(b.x, f), product(b.y, f));
    }
  }
  // x / s = (x 2^-e) / m, s = m 2^e: nothing in between leaves the range of float32
  const float to = pow2(-min((int)(__float_as_uint(s) >> 23) - 127, 126)), m = s * to;
  for (int i = t; i < n * (D / 4); i += kThreads) {
    const uint2 v = make_uint2(nan_to_0(at(i).x), nan_to_0(at(i).y));
    reinterpret_cast<uint32_t*>(page + row0 * D)[i] =
        e4m3x4(quotient(__uint_as_float(v.x << 16) * to, m), quotient(__uint_as_float(v.x & 0xffff0000u) * to, m),
               quotient(__uint_as_float(v.y << 16) * to, m), quotient(__uint_as_float(v.y & 0xffff0000u) * to, m));
  }
  if (t == 0) *scale = s;
}

// The new rows [row0, row0 + n) of one block and head, by one warp (kGroup = 1)
// or four (kGroup = 4, thread `t` of 128).  A lane holds 4 values of a row: D / 4
// lanes make a row, 128 / D rows an access.  Four warps hold up to 64 rows in
// registers: one read, many loads in flight.  One warp, for the few rows of
// single tokens and drafts, holds 8 accesses; where there are more it reads
// them twice.
template <int D, int kGroup>
__device__ __forceinline__ void store_rows(const __nv_bfloat16* __restrict__ src, int64_t stride, int row0, int n,
                                           uint8_t* __restrict__ page, float* __restrict__ scale, int t, int bar,
                                           uint32_t* __restrict__ shared_max) {
  constexpr int kRowsPer = 128 / D;
  constexpr int kHeld = kGroup == 4 ? kBlock / 4 / kRowsPer : 8;  // accesses
  const int lane = t & 31, warp = t >> 5, sub = lane / (D / 4), col = 4 * (lane % (D / 4));
  const float old = row0 > 0 ? *scale : 0.f;
  // Whether the block goes the other way (the same for the group): known before the rows are read, or, by the one
  // warp that waits for both reads anyway, behind them (64 single tokens 2.9 us, before them 3.1).
  auto elsewhere = [&]() {
    if ((__float_as_uint(old) & 0x7fffffu) == 0u && old < INFINITY) return false;
    store_rows_any<D, kGroup>(src, stride, row0, n, page, scale, old, t, bar, shared_max);
    return true;
  };
  if (kGroup == 4 && elsewhere()) return;
  const int first = warp * kHeld * kRowsPer;  // this warp's first row
  uint2 v[kHeld];
  // The largest magnitude's bits: as integers, and again without infinities and NaN where there are any (`special`,
  // the same for the group: most blocks need neither that nor NaN made 0, a third of the work).
  auto amax = [&](bool finite) {
    uint32_t top = 0u;
    for (int base = first; base < n; base += kGroup == 4 ? kBlock : kHeld * kRowsPer) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int r = base + i * kRowsPer + sub;
        if (kGroup == 4 && finite) break;  // (held)
        v[i] = r < n ? __ldg(reinterpret_cast<const uint2*>(src + r * stride + col)) : make_uint2(0u, 0u);
      }
      if (finite) {
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          most = finite_amax(finite_amax(most, v[i].x), v[i].y);
          v[i] = make_uint2(nan_to_0(v[i].x), nan_to_0(v[i].y));
        }
        top = max(top, __float_as_uint(most));  // non-negative: ordered as its bits
      } else {
        uint32_t pair = 0u;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) pair = max_u16x2(pair, max_u16x2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu));
        top = max(top, max(pair << 16, pair & 0xffff0000u));
      }
    }
    top = __reduce_max_sync(kAll, top);
    if (kGroup == 4) {
      if (lane == 0) shared_max[warp] = top;
      named_bar_sync(bar, 128);  // and every warp has read the old scale
      top = max(max(shared_max[0], shared_max[1]), max(shared_max[2], shared_max[3]));
    }
    return top;
  };
  uint32_t top = amax(false);
  if (kGroup == 1 && elsewhere()) return;
  const bool special = top >= 0x7f800000u;
  if (special) {
    if (kGroup == 4) named_bar_sync(bar, 128);  // shared_max has been read
    top = amax(true);
  }
  float s, inv;
  block_scale(old, top, s, inv);
  if (row0 > 0 && old < s) rescale_codes(reinterpret_cast<uint32_t*>(page), row0 * (D / 4), old * inv, t, 32 * kGroup);
  uint8_t* dst = page + (row0 + sub) * D + col;
  const bool again = kGroup == 1 && n > kHeld * kRowsPer;
  for (int base = first; base < n; base += kGroup == 4 ? kBlock : kHeld * kRowsPer) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int r = base + i * kRowsPer + sub;
      if (r >= n) break;
      if (again) v[i] = __ldg(reinterpret_cast<const uint2*>(src + r * stride + col));
      if (again && special) v[i] = make_uint2(nan_to_0(v[i].x), nan_to_0(v[i].y));
      *reinterpret_cast<uint32_t*>(dst + (base + i * kRowsPer) * D) = codes_of(v[i], inv);
    }
  }
  if (t == 0) *scale = s;
}

template <int D, int kGroup>
__global__ void __launch_bounds__(32 * kStoreWarps, 4) kv_store_kernel(const __grid_constant__ KvStoreArgs a) {
  __shared__ uint32_t group_max[kStoreWarps];
  const int u = (int)blockIdx.x, group = (int)threadIdx.x / (32 * kGroup), t = (int)threadIdx.x % (32 * kGroup);
  const int item = (int)blockIdx.y * (kStoreWarps / kGroup) + group;
  if (item >= 2 * a.HK) return;
  // request r's units start at floor(query_start_r / 64) + 2 r
  const int r = search_units(a.R, u, [&](int i) { return clamp_start(a.query_start, i, a.T) / kBlock + 2 * i; });
  const int t0 = clamp_start(a.query_start, r, a.T), t1 = clamp_start(a.query_start, r + 1, a.T);
  const int local = u - (t0 / kBlock + 2 * r);
  const int64_t len = a.seq_lens[r], ctx = len - (t1 - t0);
  if (t1 <= t0 || ctx < 0 || local < 0) return;
  const int64_t j = ctx / kBlock + local;  // logical block
  if (j * kBlock >= len || j >= a.MB) return;
  const int b = __ldg(a.block_table + (int64_t)r * a.MB + j);
  if (b < 0 || b >= a.NB) return;
  const int64_t p0 = max(ctx, j * kBlock), p1 = min(len, (j + 1) * kBlock);
  const int row0 = (int)(p0 % kBlock), n = (int)(p1 - p0);
  const int h = item >> 1;
  const bool is_v = item & 1;
  const int64_t bh = (int64_t)b * a.HK + h;
  const __nv_bfloat16* src = is_v ? static_cast<const __nv_bfloat16*>(a.v) + (t0 + (p0 - ctx)) * a.v_stride
                                  : static_cast<const __nv_bfloat16*>(a.k) + (t0 + (p0 - ctx)) * a.k_stride;
  src += (int64_t)h * D;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  uint8_t* page = (is_v ? a.v_cache : a.k_cache) + bh * (kBlock * D);
  float* scale = (is_v ? a.v_scale : a.k_scale) + bh;
  store_rows<D, kGroup>(src, stride, row0, n, page, scale, t, 1 + group, group_max + 4 * group);
}

}  // namespace

template <int D, int kGroup>
static void launch(const KvStoreArgs& a, cudaStream_t stream) {
  constexpr int kItems = kStoreWarps / kGroup;
  const dim3 grid((unsigned)(a.T / kBlock + 2 * a.R), (unsigned)((2 * a.HK + kItems - 1) / kItems));
  kv_store_kernel<D, kGroup><<<grid, 32 * kStoreWarps, 0, stream>>>(a);
}

cudaError_t launch_kv_store(const KvStoreArgs& a, cudaStream_t stream) {
  // Four warps a block and head where a request brings 16 rows or more on average: one warp | four take 2.9 | 5.2 us
  // for 64 requests of one row, 14.1 | 12.6 for 200 of 9 on average (38 of them of 20 to 60), 21.2 | 7.6 for 64 of 34
  // on average (8 heads, D = 128).
  const bool many = a.T / 16 >= a.R;
  if (a.D == 128)
    many ? launch<128, 4>(a, stream) : launch<128, 1>(a, stream);
  else
    many ? launch<64, 4>(a, stream) : launch<64, 1>(a, stream);
  return cudaGetLastError();
}

}  // namespace smla
