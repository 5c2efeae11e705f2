// Attention of a ragged batch over the paged 8-bit K/V cache.
//
// For token t (position p of its request r) and head h of K/V head g = h / G,
// over the keys j of the request that t sees, lo <= j < hi,
//   hi = min(seq_len_r, max(p + 1, prefix_r)),
//   lo = max(0, p - window + 1 if window > 0, doc_start_t),
//   x_j = sm_scale * <q[t,h,:], codes_K(j)> * k_scale(block of j, g)
//   x_j = softcap * tanh(x_j / softcap)   if softcap > 0
//   x_j = x_j - slope_h |p - j|           with slopes
//   out = sum_j softmax(x)_j codes_V(j) v_scale(block of j, g), lse = log sum_j exp(x_j);
// a token that sees no key gets out = 0, lse = -inf.  Keys of a block whose
// table entry is outside [0, NB) are not seen.
//
// This kernel takes up to N rows (tokens x heads of one K/V head) per query
// tile, N = 16 or 32: single tokens and short drafts.  Each key is read once
// and meets few rows, so HBM bounds it, and the design keeps the codes moving
// from HBM to the tensor cores with no instruction spent on them:
//  * A key tile is 128 keys, two blocks; TMA copies each block's 64 x D codes
//    of the head (contiguous in the cache) into a ring of stages.
//  * Both products run on the codes as stored (tcgen05 kind::f8f6f4), keys or
//    value columns in the MMA's 128 rows, the query rows in its N columns:
//      S^T[key, row] = K Q^T, q split into two e4m3 terms, q 2^s = hi + lo
//        (s puts the row's largest near 448), exact for components down to
//        2^-10 of it: q has 8 significant bits, and hi leaves at most 4;
//      O^T[d, row] = V^T P^T per block, P in an e4m3 term and an e5m2 term of
//        the remainder (about 8 significant bits where P > 2^-14, and down to
//        2^-23 of the largest weight: many small weights keep their sum).
//  * Softmax: thread = key, N columns; the block's K scale folds into the
//    logit.  P = 2^(x - m'), m' a running reference per row that is refreshed
//    (to put the tile's maximum at 2^6.25) only when a tile exceeds 2^8.75, so
//    a tile usually costs one vote of the warps instead of N maxima.
//  * O^T of each tile is read from tensor memory and added, times the block's
//    V scale, to sums in registers: no rescaling pass, any scales.
//  * The key tiles of the whole call form one sequence (smla_paged.cuh) that
//    the persistent CTAs share equally, whatever the lengths; a unit that
//    several CTAs share is merged by a second kernel.  Lengths are read on the
//    device only.
//  * Roles: TMA producer, QK^T issuer, P.V issuer, scheduler (segments ahead,
//    their Q split and columns), N / 16 groups of 4 softmax warps, 4 warps
//    that sum O.
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
#include "smla_paged.cuh"

namespace smla {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kTop = 8.75f;      // P = 2^(x - m') <= 2^8.75 < 430 (e4m3: 448)
constexpr float kRefresh = 6.25f;  // a refreshed m' puts the tile's maximum at 2^6.25
constexpr float kNoMax = -3e38f;   // m' of a row that has seen nothing

__host__ __device__ constexpr uint32_t idesc_f8(uint32_t M, uint32_t N, uint32_t b_e5m2, uint32_t a_mn, uint32_t b_mn) {
  return (1u << 4) | (b_e5m2 << 10) | (a_mn << 15) | (b_mn << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
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
__device__ __forceinline__ float warp_max(float x) {  // through an order-preserving map to integers; no NaN
  int k = __float_as_int(x);
  k = __reduce_max_sync(kAll, k >= 0 ? k : k ^ 0x7FFFFFFF);
  return __int_as_float(k >= 0 ? k : k ^ 0x7FFFFFFF);
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
// Two weights -> e4m3 codes and e5m2 codes of the remainders (low byte from
// x0).  The split runs in f16x2: 11 bits, more than the two terms keep.
__device__ __forceinline__ void split_p(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  uint32_t a, d, r;
  uint16_t t;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(a) : "f"(x1), "f"(x0));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(t) : "r"(a));
  hi = t;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(t));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(d));
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(t) : "r"(r));
  lo = t;
}
// Offset of 16-byte chunk ch of row r, rows of D bytes under the D-byte swizzle.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int ch) {
  return (uint32_t)(r * D + ((D == 128 ? ch ^ (r & 7) : ch ^ ((r >> 1) & 3)) << 4));
}

struct Params {
  PagedAttnArgs a;
  // Rows of a query tile: tq tokens x up to Gr of the G heads of a K/V head; more than N heads are cut into
  // `cuts` groups, which the sequence of units counts as K/V heads of their own (HV = HK * cuts).
  int G, Gr, cuts, HV, tq;
  int ctas;
  int* status;
  PagedMerge* merge;    // [ctas]
  float* part_ml;       // [2 ctas][m' | l][N]
  float* part_o;        // [2 ctas][N][D]
};

// What a row (column of the MMAs) needs of its own.
template <int N>
struct Columns {
  float scale[N];  // logit = S * scale * k_scale, in log2 units (natural ones with softcap)
  float slope[N];  // log2 units per key of distance
  int pos[N], lo[N], hi[N];
};

template <int D, int N>
struct Lay {
  static constexpr int kHalves = N / 16;  // softmax groups
  static constexpr int kWarps = 4 + 4 * kHalves + 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPerSm = N == 16 ? 2 : 1;
  static constexpr int kKTile = kKeyTile * D;
  static constexpr int kStage = 2 * kKTile;
  static constexpr int kStages = (N == 16 ? 3 : 5) * (128 / D);
  static constexpr int kMeta = kStages + 2;        // ring of page scales and flags
  static constexpr int kQTerm = N * D;             // one term of Q
  static constexpr int kQBuf = 2 * kQTerm;
  static constexpr int kSegs = 2;
  static constexpr int kP = kKeyTile * 2 * N;
  static constexpr int kRefs = 4;                  // ring of (m', v scales) towards the summing warps
  static constexpr int kOffQ = kStages * kStage;
  static constexpr int kOffP = kOffQ + kSegs * kQBuf;
  static constexpr int kOffCols = kOffP + kP;
  static constexpr int kOffMeta = kOffCols + kSegs * (int)sizeof(Columns<N>);
  static constexpr int kOffRefs = kOffMeta + kMeta * 32;
  static constexpr int kRef = N * 4 + 16;          // m'[N], v scales, change flag
  static constexpr int kOffRed = kOffRefs + kRefs * kRef;          // float [halves][4][16]
  static constexpr int kOffSum = kOffRed + kHalves * 4 * 16 * 4;   // float [halves][4][16]
  static constexpr int kOffFin = kOffSum + kHalves * 4 * 16 * 4;   // float [2][m' | l][N]
  static constexpr int kOffSeg = kOffFin + 2 * 2 * N * 4;
  static constexpr int kOffBar = (kOffSeg + kSegs * (int)sizeof(Segment) + 7) / 8 * 8;
  enum {
    kKFull = 0, kVFull = kKFull + kStages, kEmpty = kVFull + kStages, kSFull = kEmpty + kStages, kSFree = kSFull + 2,
    kPFull = kSFree + 2, kPFree, kOFull, kOFree = kOFull + 2, kRefFull = kOFree + 2, kSegFull = kRefFull + kRefs,
    kSegFree = kSegFull + kSegs, kFinFull = kSegFree + kSegs, kDrainQk = kFinFull + 2, kDrainPv, kNumBars
  };
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmem = kOffMisc + 16 + 1024;
  static constexpr int kTmemS = 0, kTmemO = 2 * N;  // S [2][N], O [2][2 blocks][N]
  static constexpr int kTmemCols = N == 16 ? 128 : 256;
  static_assert(kTmemO + 4 * N <= kTmemCols, "tensor memory");
  static_assert(kPerSm * (kSmem + 1024) <= 233472, "shared memory of an SM");
  static_assert(kStage % 1024 == 0 && kQTerm % 512 == 0 && kOffP % 128 == 0 && kOffCols % 16 == 0 &&
                kOffRefs % 16 == 0 && kRef % 16 == 0 && kOffFin % 16 == 0 && kOffRed % 16 == 0, "alignment");
  static_assert((kMaxPagedRequests + 1 + kWarps) * 8 <= kStages * kStage, "prefix sums fit the stages");
};

// Tiles of request r (over its query tiles and the K/V heads).
__device__ __forceinline__ int64_t request_tiles(const Params& p, int r) {
  PagedRequest q;
  q.load(p.a, r);
  int64_t n = 0;
  for (int t = q.t0; t < q.t1; t += p.tq) {
    int lo, hi, al, ah, first, count;
    q.range(p.a, t, min(t + p.tq, q.t1), lo, hi, al, ah);
    key_tiles(lo, hi, first, count);
    n += count;
  }
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

template <int D, int N>
__global__ void __launch_bounds__(Lay<D, N>::kThreads, Lay<D, N>::kPerSm)
    paged_attn_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map) {
  using L = Lay<D, N>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  grid_launch_dependents();  // the merge may be launched behind this grid; it waits for the grid's end
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedAttnArgs& a = p.a;

  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&bars[L::kKFull + i], 1);
      mbar_init(&bars[L::kVFull + i], 1);
      mbar_init(&bars[L::kEmpty + i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[L::kSFull + i], 1);
      mbar_init(&bars[L::kSFree + i], 4 * L::kHalves);
      mbar_init(&bars[L::kOFull + i], 1);
      mbar_init(&bars[L::kOFree + i], 4);
      mbar_init(&bars[L::kFinFull + i], L::kHalves);
    }
    mbar_init(&bars[L::kPFull], 4 * L::kHalves);
    mbar_init(&bars[L::kPFree], 1);
    for (int i = 0; i < L::kRefs; ++i) mbar_init(&bars[L::kRefFull + i], L::kHalves);
    for (int i = 0; i < L::kSegs; ++i) {
      mbar_init(&bars[L::kSegFull + i], 1);
      mbar_init(&bars[L::kSegFree + i], 1 + 1 + 4 * L::kHalves + 4);
    }
    mbar_init(&bars[L::kDrainQk], 1);
    mbar_init(&bars[L::kDrainPv], 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 3) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  // prefix sums of the requests' tiles, in the stages' memory (before any copy lands there)
  int64_t* prefix = reinterpret_cast<int64_t*>(smem);
  for (int r = tid; r < a.R; r += L::kThreads) prefix[r] = request_tiles(p, r);
  __syncthreads();
  scan_tiles<L::kThreads>(prefix, a.R);
  const int64_t total = prefix[a.R];
  // with fewer tiles than CTAs the first CTAs take one each: a unit's parts are consecutive CTAs
  const int ctas = (int)min((int64_t)p.ctas, total);
  const bool idle = (int)blockIdx.x >= ctas;
  const int64_t x0 = idle ? 0 : range_begin(blockIdx.x, total, ctas);
  const int64_t x1 = idle ? 0 : range_begin((int64_t)blockIdx.x + 1, total, ctas);
  const int n_local = (int)(x1 - x0);
  int r0 = 0;
  int64_t off0 = 0;
  if (warp == 2 && n_local > 0) {  // the request of this CTA's first tile
    int hi = a.R;
    while (hi - r0 > 1) {
      const int mid = (r0 + hi) >> 1;
      if (prefix[mid] <= x0) r0 = mid;
      else hi = mid;
    }
    off0 = x0 - prefix[r0];
  }
  fence_proxy_async_smem();  // the copies may overwrite the prefix sums
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
#define PA_WAIT(idx, parity) mbar_wait(&bars[(idx)], (parity), abort_flag, p.status, kDevWaitTimeout)

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    const int outside = (int)(a.NB * a.HK * kBlock);  // a row behind the cache: reads as zeros
    int tl = 0, seg = 0;
    bool dead = false;
    while (tl < n_local && !dead) {
      const int sb = seg % L::kSegs;
      dead = __any_sync(kAll, !PA_WAIT(L::kSegFull + sb, (seg / L::kSegs) & 1));
      if (dead) break;
      const Segment s = *reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment));
      const int32_t* row = a.block_table + (int64_t)s.r * a.MB;
      // lane l holds block base + l of the row: its cache block (-1: none) and scales; the next 32 are
      // fetched while these are in use
      auto fetch = [&](int page, int& b, float& ks, float& vs) {
        b = -1;
        ks = vs = 0.f;
        if (page * kBlock < s.hi && (page + 1) * kBlock > s.lo) {
          const int x = __ldg(row + page);
          if (x >= 0 && x < a.NB) {
            b = x;
            ks = __ldg(a.k_scale + (int64_t)x * a.HK + s.g);
            vs = __ldg(a.v_scale + (int64_t)x * a.HK + s.g);
          }
        }
      };
      int b, nb;
      float ks, vs, nks, nvs;
      fetch(2 * s.kt + lane, b, ks, vs);
      for (int i = 0; i < s.n && !dead; ++i, ++tl) {
        const int at = (2 * i) & 31;
        if (at == 0) {
          if (i > 0) {
            b = nb;
            ks = nks;
            vs = nvs;
          }
          if (i + 16 < s.n) fetch(2 * (s.kt + i + 16) + lane, nb, nks, nvs);
        }
        const int b0 = __shfl_sync(kAll, b, at), b1 = __shfl_sync(kAll, b, at + 1);
        const float k0 = __shfl_sync(kAll, ks, at), k1 = __shfl_sync(kAll, ks, at + 1);
        const float v0 = __shfl_sync(kAll, vs, at), v1 = __shfl_sync(kAll, vs, at + 1);
        const int st = tl % L::kStages, use = tl / L::kStages;
        if (use > 0) dead = __any_sync(kAll, !PA_WAIT(L::kEmpty + st, (use + 1) & 1));
        if (dead) break;
        if (lane == 0) {
          float* meta = reinterpret_cast<float*>(smem + L::kOffMeta + (tl % L::kMeta) * 32);
          *reinterpret_cast<float4*>(meta) = make_float4(k0, k1, v0, v1);
          reinterpret_cast<int*>(meta)[4] = (b0 >= 0 ? 1 : 0) | (b1 >= 0 ? 2 : 0);
          const int y0 = b0 >= 0 ? (b0 * a.HK + s.g) * kBlock : outside;
          const int y1 = b1 >= 0 ? (b1 * a.HK + s.g) * kBlock : outside;
          const uint32_t kd = smem_u32(smem + st * L::kStage), vd = kd + L::kKTile;
          mbar_arrive_expect_tx(&bars[L::kKFull + st], L::kKTile);
          tma_load_2d(kd, &k_map, 0, y0, &bars[L::kKFull + st]);
          tma_load_2d(kd + kBlock * D, &k_map, 0, y1, &bars[L::kKFull + st]);
          mbar_arrive_expect_tx(&bars[L::kVFull + st], L::kKTile);
          tma_load_2d(vd, &v_map, 0, y0, &bars[L::kVFull + st]);
          tma_load_2d(vd + kBlock * D, &v_map, 0, y1, &bars[L::kVFull + st]);
        }
        __syncwarp();
      }
      if (lane == 0 && !dead) mbar_arrive(&bars[L::kSegFree + sb]);
      ++seg;
    }
    // no copy may still be landing when the CTA exits
    for (int j = max(0, tl - L::kStages); j < tl; ++j) {
      mbar_wait_drain(&bars[L::kKFull + j % L::kStages], (j / L::kStages) & 1);
      mbar_wait_drain(&bars[L::kVFull + j % L::kStages], (j / L::kStages) & 1);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- QK^T issuer
    if (lane == 0 && n_local > 0) {
      constexpr uint32_t id = idesc_f8(128, N, 0, 0, 0);
      constexpr uint32_t lay = D == 128 ? kLayoutSw128 : kLayoutSw64;
      const uint64_t dk0 = make_sdesc(smem_u32(smem), 16, 8 * D, lay);
      const uint64_t dq0 = make_sdesc(smem_u32(smem + L::kOffQ), 16, 8 * D, lay);
      int tl = 0, seg = 0;
      bool dead = false;
      while (tl < n_local && !dead) {
        const int sb = seg % L::kSegs;
        if (!PA_WAIT(L::kSegFull + sb, (seg / L::kSegs) & 1)) break;
        const int n = reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment))->n;
        const uint64_t dq = dq0 + (uint64_t)((sb * L::kQBuf) >> 4);
        for (int i = 0; i < n; ++i, ++tl) {
          const int st = tl % L::kStages, buf = tl & 1;
          if ((tl >= 2 && !PA_WAIT(L::kSFree + buf, ((tl >> 1) + 1) & 1)) ||
              !PA_WAIT(L::kKFull + st, (tl / L::kStages) & 1)) {
            dead = true;
            break;
          }
          tc_fence_after();
          const uint64_t dk = dk0 + (uint64_t)((st * L::kStage) >> 4);
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              mma_f8(tmem + L::kTmemS + buf * N, dk + ((32 * k) >> 4), dq + ((term * L::kQTerm + 32 * k) >> 4), id,
                     term + k > 0 ? 1u : 0u);
          mma_commit(&bars[L::kSFull + buf]);
        }
        if (!dead) mma_commit(&bars[L::kSegFree + sb]);  // the segment's Q has been read
        ++seg;
      }
      // every issued operation completes before tensor memory is released
      mma_commit(&bars[L::kDrainQk]);
      mbar_wait_drain(&bars[L::kDrainQk], 0);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---------------------------------------------------------------- P.V issuer
    if (lane == 0 && n_local > 0) {
      constexpr uint32_t id_hi = idesc_f8(128, N, 0, 1, 1), id_lo = idesc_f8(128, N, 1, 1, 1);
      // V: rows are keys, D-byte swizzle, read MN-major; at D = 64 the MMA's upper 64 rows read the same
      // columns again (atoms 0 bytes apart) and their results are not used
      const uint64_t dv0 = make_sdesc(smem_u32(smem + L::kKTile), 0, 8 * D, D == 128 ? kLayoutSw128 : kLayoutSw64);
      // P: blocks of 8 keys x 16 rows, hi blocks then lo blocks of 8 keys
      const uint64_t dp0 = make_sdesc(smem_u32(smem + L::kOffP), 16 * N, 128, kLayoutNone);
      for (int tl = 0; tl < n_local; ++tl) {
        const int st = tl % L::kStages, buf = tl & 1;
        if (!PA_WAIT(L::kPFull, tl & 1) || !PA_WAIT(L::kVFull + st, (tl / L::kStages) & 1) ||
            (tl >= 2 && !PA_WAIT(L::kOFree + buf, ((tl >> 1) + 1) & 1)))
          break;
        tc_fence_after();
        const uint64_t dv = dv0 + (uint64_t)((st * L::kStage) >> 4);
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int step = 2 * blk + k;  // 32 keys
              mma_f8(tmem + L::kTmemO + (2 * buf + blk) * N, dv + ((32 * D * step) >> 4),
                     dp0 + ((64 * N * step + term * 8 * N) >> 4), term ? id_lo : id_hi, term + k > 0 ? 1u : 0u);
            }
        mma_commit(&bars[L::kPFree]);
        mma_commit(&bars[L::kEmpty + st]);  // the tile's QK^T completed before its P was written
        mma_commit(&bars[L::kOFull + buf]);
      }
      mma_commit(&bars[L::kDrainPv]);
      mbar_wait_drain(&bars[L::kDrainPv], 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------------------------------------------------------- scheduler
    // Walks this CTA's range; for each segment: the record, the rows' columns
    // and the two terms of Q.
    PagedMerge mine{0, 0, 0, 0, 0};
    if (n_local > 0) {
      int r = r0, seg = 0;
      int64_t x = x0, off = off0;
      bool dead = false;
      while (x < x1 && r < a.R && !dead) {
        PagedRequest q;
        q.load(a, r);
        for (int ta = q.t0; ta < q.t1 && x < x1 && !dead; ta += p.tq) {
          const int tb = min(ta + p.tq, q.t1);
          Segment s;
          q.range(a, ta, tb, s.lo, s.hi, s.all_lo, s.all_hi);
          int first, count;
          key_tiles(s.lo, s.hi, first, count);
          if (s.hi <= s.lo) s.lo = s.hi = 0;  // nothing is seen: no block is read
          if (off >= (int64_t)count * p.HV) {
            off -= (int64_t)count * p.HV;
            continue;
          }
          s.r = r;
          s.t0 = ta;
          s.ntok = tb - ta;
          s.pos0 = q.pos(ta);
          for (int g = (int)(off / count); g < p.HV && x < x1; ++g) {
            const int skip = (int)(off - (int64_t)g * count);  // tiles of this unit before this CTA's range
            off = (int64_t)(g + 1) * count;
            s.g = g / p.cuts;
            s.h0 = s.g * p.G + g % p.cuts * p.Gr;
            s.heads = min(p.Gr, p.G - g % p.cuts * p.Gr);
            s.kt = first + skip;
            s.n = (int)min((int64_t)(count - skip), x1 - x);
            const bool ends = skip + s.n == count;
            s.slot = skip == 0 ? (ends ? -1 : 1) : 0;
            s.parts = 0;
            if (s.slot == 1) {
              s.parts = range_of(x + count - 1, total, ctas) - (int)blockIdx.x + 1;
              mine = PagedMerge{ta, s.ntok, s.h0, s.heads, s.parts};
            }
            x += s.n;
            const int sb = seg % L::kSegs;
            if (seg >= L::kSegs) dead = __any_sync(kAll, !PA_WAIT(L::kSegFree + sb, (seg / L::kSegs + 1) & 1));
            if (dead) break;
            if (lane == 0) *reinterpret_cast<Segment*>(smem + L::kOffSeg + sb * sizeof(Segment)) = s;
            Columns<N>* cols = reinterpret_cast<Columns<N>*>(smem + L::kOffCols + sb * sizeof(Columns<N>));
            const int rows = s.ntok * s.heads;
            if (lane < N) {
              const int t = min(ta + lane / s.heads, tb - 1), h = s.h0 + lane % s.heads;
              cols->pos[lane] = q.pos(t);
              cols->lo[lane] = lane < rows ? q.lo(a, t) : 0;
              cols->hi[lane] = lane < rows ? q.hi(t) : 0;
              cols->slope[lane] = a.alibi_slopes && lane < rows ? __ldg(a.alibi_slopes + h) * kLog2e : 0.f;
            }
            // D / 8 lanes per row, 8 values each
            constexpr int kLanes = D / 8, kRowsPer = 32 / kLanes;
            const uint32_t qd = smem_u32(smem + L::kOffQ + sb * L::kQBuf);
            const int sub = lane / kLanes, c = lane % kLanes;
#pragma unroll 4
            for (int i = 0; i < N / kRowsPer; ++i) {
              const int row = i * kRowsPer + sub;
              uint4 v = make_uint4(0u, 0u, 0u, 0u);
              if (row < rows)
                v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                         (int64_t)(ta + row / s.heads) * a.q_stride +
                                                         (int64_t)(s.h0 + row % s.heads) * D) + c);
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
              uint32_t amax = 0u;  // of the magnitudes' bits
#pragma unroll
              for (int k = 0; k < 4; ++k) amax = max(amax, max((w[k] << 16) & 0x7fffffffu, w[k] & 0x7fff0000u));
#pragma unroll
              for (int o = 1; o < kLanes; o <<= 1) amax = max(amax, __shfl_xor_sync(kAll, amax, o));
              // 2^sh: amax = (1 + f) 2^e to at most 448 = 1.75 * 2^8
              int sh = 8 - ((int)(amax >> 23) - 127) - ((amax & 0x7fffffu) > 0x600000u);
              sh = amax == 0u ? 0 : min(sh, 120);
              const float f = __uint_as_float((uint32_t)(sh + 127) << 23);
              uint32_t hi[2] = {0u, 0u}, lo[2] = {0u, 0u};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float y0 = __uint_as_float(w[k] << 16) * f, y1 = __uint_as_float(w[k] & 0xffff0000u) * f;
                const uint32_t hc = e4m3x2(y0, y1);
                const float2 back = e4m3x2_f32(hc);
                hi[k >> 1] |= hc << (16 * (k & 1));
                lo[k >> 1] |= e4m3x2(y0 - back.x, y1 - back.y) << (16 * (k & 1));
              }
              const uint32_t dst = qd + swz<D>(row, c >> 1) + 8 * (c & 1);
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst), "r"(hi[0]), "r"(hi[1]) : "memory");
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst + L::kQTerm), "r"(lo[0]), "r"(lo[1]) : "memory");
              if (c == 0) {
                // a row with an infinity or NaN has no finite result
                const float back = amax >= 0x7f800000u ? __uint_as_float(0x7fc00000u)
                                                       : __uint_as_float((uint32_t)(127 - sh) << 23);
                cols->scale[row] = a.sm_scale * back * (a.softcap > 0.f ? 1.f : kLog2e);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[L::kSegFull + sb]);
            ++seg;
          }
          off = 0;
        }
        ++r;
      }
    }
    if (lane == 0) p.merge[blockIdx.x] = mine;
  } else if (warp < 4 + 4 * L::kHalves) {
    // ---------------------------------------------------------------- softmax: thread = key, 16 rows per group
    const int half = (warp - 4) >> 2, quarter = warp & 3;
    const int key = 32 * quarter + lane;
    const uint32_t s_addr = tmem + ((uint32_t)(32 * quarter) << 16) + L::kTmemS + 16 * half;
    const uint32_t p_addr = smem_u32(smem + L::kOffP) + (key >> 3) * 16 * N + (key & 7) * 16 + half * 128;
    float* red = reinterpret_cast<float*>(smem + L::kOffRed) + half * 64;
    float* sums = reinterpret_cast<float*>(smem + L::kOffSum) + half * 64;
    const int bar = 1 + half;
    int tl = 0, seg = 0;
    bool dead = false;
    auto wait = [&](int idx, uint32_t parity) {  // `dead` stays the same in the whole warp
      if (!dead) dead = !PA_WAIT(idx, parity);
      dead = __any_sync(kAll, dead);
    };
    while (tl < n_local && !dead) {
      const int sb = seg % L::kSegs;
      wait(L::kSegFull + sb, (seg / L::kSegs) & 1);
      if (dead) break;
      const Segment* sp = reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment));
      const Columns<N>* cols = reinterpret_cast<const Columns<N>*>(smem + L::kOffCols + sb * sizeof(Columns<N>));
      const int kt = sp->kt, n = sp->n, lo = sp->lo, hi = sp->hi, all_lo = sp->all_lo, all_hi = sp->all_hi;
      float m[16], l[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        m[c] = kNoMax;
        l[c] = 0.f;
      }
      for (int i = 0; i < n; ++i, ++tl) {
        const int buf = tl & 1, st = tl % L::kStages;
        wait(L::kKFull + st, (tl / L::kStages) & 1);  // the tile's scales and flags
        wait(L::kSFull + buf, (tl >> 1) & 1);
        if (dead) break;
        tc_fence_after();
        uint32_t raw[16];
        tmem_ld16_sync(s_addr + buf * N, raw);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kSFree + buf]);
        const float* meta = reinterpret_cast<const float*>(smem + L::kOffMeta + (tl % L::kMeta) * 32);
        const float ks = meta[key >> 6];
        const int pages = reinterpret_cast<const int*>(meta)[4];
        const int j0 = (kt + i) * kKeyTile, j = j0 + key;
        float x[16];
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) {
          const float4 f = *reinterpret_cast<const float4*>(&cols->scale[16 * half + 4 * c4]);
          x[4 * c4] = __uint_as_float(raw[4 * c4]) * f.x * ks;
          x[4 * c4 + 1] = __uint_as_float(raw[4 * c4 + 1]) * f.y * ks;
          x[4 * c4 + 2] = __uint_as_float(raw[4 * c4 + 2]) * f.z * ks;
          x[4 * c4 + 3] = __uint_as_float(raw[4 * c4 + 3]) * f.w * ks;
        }
        if (a.softcap > 0.f) {
          // cap tanh(x / cap) = cap (1 - 2 / (1 + e^(2 x / cap))), to within a few 2^-23 cap
          const float to = 2.f * kLog2e / a.softcap, cap = a.softcap * kLog2e;
#pragma unroll
          for (int c = 0; c < 16; ++c) x[c] = fmaf(-2.f * cap, __fdividef(1.f, 1.f + ex2_approx(x[c] * to)), cap);
        }
        if (a.alibi_slopes) {
#pragma unroll
          for (int c = 0; c < 16; ++c)
            x[c] = fmaf(-cols->slope[16 * half + c], fabsf((float)(cols->pos[16 * half + c] - j)), x[c]);
        }
        const bool inside = j0 >= all_lo && j0 + kKeyTile <= all_hi && pages == 3;
        if (!inside) {
          const bool page_ok = (pages >> (key >> 6)) & 1;
#pragma unroll
          for (int c = 0; c < 16; ++c)
            if (!page_ok || j < cols->lo[16 * half + c] || j >= cols->hi[16 * half + c]) x[c] = -INFINITY;
        }
        float over = -INFINITY;
#pragma unroll
        for (int c = 0; c < 16; ++c) over = fmaxf(over, x[c] - m[c]);
        const bool refresh = bar_any(bar, 128, over > kTop);
        if (refresh) {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float mx = warp_max(x[c] == x[c] ? x[c] : -INFINITY);
            if (lane == c) red[quarter * 16 + c] = mx;
          }
          named_bar_sync(bar, 128);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float mx = fmaxf(fmaxf(red[c], red[16 + c]), fmaxf(red[32 + c], red[48 + c]));
            if (mx - m[c] > kTop) {
              const float to = mx - kRefresh;
              l[c] *= ex2_approx(m[c] - to);
              m[c] = to;
            }
          }
        }
        uint32_t hw[8], lw[8];
#pragma unroll
        for (int c2 = 0; c2 < 8; ++c2) {
          const float p0 = ex2_approx(x[2 * c2] - m[2 * c2]), p1 = ex2_approx(x[2 * c2 + 1] - m[2 * c2 + 1]);
          l[2 * c2] += p0;
          l[2 * c2 + 1] += p1;
          split_p(p0, p1, hw[c2], lw[c2]);
        }
        // the references go to the summing warps: slot tl % 4 was read before P.V of tile tl - 2 could be issued
        uint8_t* ref = smem + L::kOffRefs + (tl % L::kRefs) * L::kRef;
        if (tl > 0) wait(L::kPFree, (tl + 1) & 1);  // P.V of the previous tile has read P
        // keys that no row sees may hold any codes: their V rows become zeros
        const bool zero_v = half == 0 && (j < lo || j >= hi);
        if (__any_sync(kAll, zero_v)) wait(L::kVFull + st, (tl / L::kStages) & 1);
        if (dead) break;
        if (quarter == 0 && lane < 16 && (refresh || i == 0)) {
#pragma unroll
          for (int c = 0; c < 16; ++c)
            if (lane == c) reinterpret_cast<float*>(ref)[16 * half + c] = m[c];
        }
        if (quarter == 0 && lane == 0) {
          reinterpret_cast<int*>(ref)[N + 2 + half] = refresh || i == 0;
          if (half == 0) *reinterpret_cast<float2*>(ref + 4 * N) = make_float2(meta[2], meta[3]);
        }
        st_shared_v4(p_addr, hw[0] | (hw[1] << 16), hw[2] | (hw[3] << 16), hw[4] | (hw[5] << 16), hw[6] | (hw[7] << 16));
        st_shared_v4(p_addr + 8 * N, lw[0] | (lw[1] << 16), lw[2] | (lw[3] << 16), lw[4] | (lw[5] << 16),
                     lw[6] | (lw[7] << 16));
        if (zero_v) {
          const uint32_t v = smem_u32(smem + st * L::kStage + L::kKTile) + key * D;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) st_shared_v4(v + 16 * k, 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars[L::kPFull]);
          if (quarter == 0) mbar_arrive(&bars[L::kRefFull + tl % L::kRefs]);
        }
      }
      if (dead) break;
      // the rows' sums over the segment's keys
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        float v = l[c];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
        if (lane == c) sums[quarter * 16 + c] = v;
      }
      named_bar_sync(bar, 128);
      if (quarter == 0) {
        float* fin = reinterpret_cast<float*>(smem + L::kOffFin + (seg & 1) * 2 * N * 4) + 16 * half;
#pragma unroll
        for (int c = 0; c < 16; ++c)
          if (lane == c) {
            fin[c] = m[c];
            fin[N + c] = (sums[c] + sums[16 + c]) + (sums[32 + c] + sums[48 + c]);
          }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kFinFull + (seg & 1)]);
      }
      if (lane == 0) mbar_arrive(&bars[L::kSegFree + sb]);
      ++seg;
    }
  } else {
    // ---------------------------------------------------------------- sums of O: thread = value column, N rows
    const int quarter = warp & 3, d = 32 * quarter + lane;
    const uint32_t o_addr = tmem + ((uint32_t)(32 * quarter) << 16) + L::kTmemO;
    int tl = 0, seg = 0;
    bool dead = false;
    auto wait = [&](int idx, uint32_t parity) {
      if (!dead) dead = !PA_WAIT(idx, parity);
      dead = __any_sync(kAll, dead);
    };
    while (tl < n_local && !dead) {
      const int sb = seg % L::kSegs;
      wait(L::kSegFull + sb, (seg / L::kSegs) & 1);
      if (dead) break;
      const Segment s = *reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment));
      float acc[N], m[N];
#pragma unroll
      for (int c = 0; c < N; ++c) {
        acc[c] = 0.f;
        m[c] = kNoMax;
      }
      for (int i = 0; i < s.n; ++i, ++tl) {
        const int buf = tl & 1;
        wait(L::kRefFull + tl % L::kRefs, (tl / L::kRefs) & 1);
        const uint8_t* ref = smem + L::kOffRefs + (tl % L::kRefs) * L::kRef;
        const float2 vs = *reinterpret_cast<const float2*>(ref + 4 * N);
#pragma unroll
        for (int half = 0; half < L::kHalves; ++half)
          if (reinterpret_cast<const int*>(ref)[N + 2 + half]) {
#pragma unroll
            for (int c = 16 * half; c < 16 * half + 16; ++c) {
              const float to = reinterpret_cast<const float*>(ref)[c];
              acc[c] *= ex2_approx(m[c] - to);
              m[c] = to;
            }
          }
        wait(L::kOFull + buf, (tl >> 1) & 1);
        if (dead) break;
        tc_fence_after();
#pragma unroll
        for (int half = 0; half < L::kHalves; ++half) {
          uint32_t o0[16], o1[16];
          tmem_ld16(o_addr + 2 * buf * N + 16 * half, o0);
          tmem_ld16(o_addr + (2 * buf + 1) * N + 16 * half, o1);
          tmem_ld_wait();
          reg_fence16(o0);
          reg_fence16(o1);
#pragma unroll
          for (int c = 0; c < 16; ++c)
            acc[16 * half + c] = fmaf(__uint_as_float(o0[c]), vs.x,
                                      fmaf(__uint_as_float(o1[c]), vs.y, acc[16 * half + c]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kOFree + buf]);
      }
      wait(L::kFinFull + (seg & 1), (seg >> 1) & 1);
      if (dead) break;
      const float* fin = reinterpret_cast<const float*>(smem + L::kOffFin + (seg & 1) * 2 * N * 4);
      const int rows = s.ntok * s.heads;
      if (s.slot < 0) {
#pragma unroll
        for (int c = 0; c < N; ++c) {
          if (c >= rows) break;
          const float l = fin[N + c], inv = l == 0.f ? 0.f : 1.f / l;
          const int64_t row = (int64_t)(s.t0 + c / s.heads) * a.H + s.h0 + c % s.heads;
          if (D == 128 || d < D) static_cast<__nv_bfloat16*>(a.out)[row * D + d] = __float2bfloat16(acc[c] * inv);
          if (d == 0) a.lse[row] = l == 0.f ? -INFINITY : (fin[c] + log2f(l)) * kLn2;
        }
      } else {
        const int64_t part = 2 * (int64_t)blockIdx.x + s.slot;
        float* o = p.part_o + part * N * D;
#pragma unroll
        for (int c = 0; c < N; ++c) {
          if (c >= rows) break;
          if (D == 128 || d < D) o[c * D + d] = acc[c];
        }
        if (d < 2 * N) p.part_ml[part * 2 * N + d] = fin[d];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[L::kSegFree + sb]);
      ++seg;
    }
  }
#undef PA_WAIT
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// The units that several CTAs share: out = sum_i w_i O_i / sum_i w_i l_i, w_i =
// 2^(m_i - max m), lse = max m + log2 of the latter sum.  One CTA per CTA that
// began such a unit and group of rows; thread = value column.
template <int D, int N>
__global__ void __launch_bounds__(D) paged_merge_kernel(const __grid_constant__ Params p) {
  grid_dependency_wait();
  const PagedMerge u = p.merge[blockIdx.x];
  if (u.parts == 0) return;
  const int d = threadIdx.x, rows = u.ntok * u.heads;
  // the parts: slot 1 of this CTA, then slot 0 of the following ones
  auto part = [&](int i) { return i == 0 ? 2 * (int64_t)blockIdx.x + 1 : 2 * ((int64_t)blockIdx.x + i); };
  for (int c = blockIdx.y; c < rows; c += gridDim.y) {
    float top = kNoMax;
    for (int i = 0; i < u.parts; ++i) top = fmaxf(top, p.part_ml[part(i) * 2 * N + c]);
    float sum = 0.f, acc = 0.f;
#pragma unroll 4
    for (int i = 0; i < u.parts; ++i) {
      const float* ml = p.part_ml + part(i) * 2 * N + c;
      const float w = ex2_approx(ml[0] - top);
      sum = fmaf(w, ml[N], sum);
      acc = fmaf(w, p.part_o[part(i) * N * D + c * D + d], acc);
    }
    const int64_t row = (int64_t)(u.t0 + c / u.heads) * p.a.H + u.h0 + c % u.heads;
    static_cast<__nv_bfloat16*>(p.a.out)[row * D + d] = __float2bfloat16(sum == 0.f ? 0.f : acc / sum);
    if (d == 0) p.a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
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

struct Sizes {
  int ctas;
  size_t merge, ml, o, bytes;  // offsets in the workspace, and its size
};
Sizes sizes(int N, int D, int num_sms) {
  Sizes s;
  s.ctas = num_sms * (N == 16 ? 2 : 1);
  s.merge = kWsStatusBytes;
  s.ml = s.merge + align256(sizeof(PagedMerge) * s.ctas);
  s.o = s.ml + align256((size_t)2 * s.ctas * 2 * N * 4);
  s.bytes = s.o + (size_t)2 * s.ctas * N * D * 4;
  return s;
}

template <int D, int N>
cudaError_t launch(const PagedAttnArgs& a, const Sizes& sz, cudaStream_t stream) {
  using L = Lay<D, N>;
  CUtensorMap k_map, v_map;
  const int64_t rows = a.NB * a.HK * kBlock;
  cudaError_t e = cache_map(&k_map, a.k_cache, rows, D);
  if (e == cudaSuccess) e = cache_map(&v_map, a.v_cache, rows, D);
  if (e != cudaSuccess) return e;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  Params p{};
  p.a = a;
  p.G = a.H / a.HK;
  p.cuts = (p.G + N - 1) / N;
  p.Gr = (p.G + p.cuts - 1) / p.cuts;
  p.HV = a.HK * p.cuts;
  p.tq = std::max(1, N / p.Gr);
  p.ctas = sz.ctas;
  p.status = reinterpret_cast<int*>(ws);
  p.merge = reinterpret_cast<PagedMerge*>(ws + sz.merge);
  p.part_ml = reinterpret_cast<float*>(ws + sz.ml);
  p.part_o = reinterpret_cast<float*>(ws + sz.o);
  e = cudaFuncSetAttribute(paged_attn_kernel<D, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  paged_attn_kernel<D, N><<<(unsigned)p.ctas, L::kThreads, L::kSmem, stream>>>(p, k_map, v_map);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.ctas, 4);
  cfg.blockDim = dim3(D);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, N>, p);
}

}  // namespace

// N = 32 where 16 rows cannot hold the heads or the estimated tokens of a request: keys are then read
// once for up to 32 rows.
static int rows_for(int G, int max_query_len) { return (int64_t)G * std::max(1, max_query_len) <= 16 ? 16 : 32; }

size_t paged_attention_workspace(int G, int D, int max_query_len, int num_sms) {
  return sizes(rows_for(G, max_query_len), D, num_sms).bytes;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, int max_query_len, int num_sms, cudaStream_t stream) {
  const int N = rows_for(a.H / a.HK, max_query_len);
  const Sizes sz = sizes(N, a.D, num_sms);
  if (N == 16) return a.D == 128 ? launch<128, 16>(a, sz, stream) : launch<64, 16>(a, sz, stream);
  return a.D == 128 ? launch<128, 32>(a, sz, stream) : launch<64, 32>(a, sz, stream);
}

}  // namespace smla
