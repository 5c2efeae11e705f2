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
// This kernel takes up to C rows (tokens x heads of one K/V head) per query
// tile, C = 8 or 16: single tokens and short drafts.  A key is read once for up
// to C rows (17 to 48 rows of a request are two or three tiles), so HBM bounds it, and the design keeps the codes moving
// from HBM to the tensor cores with no instruction spent on them:
//  * A key tile is 128 keys, two blocks; TMA copies each block's 64 x D codes
//    of the head (contiguous in the cache) into a ring of stages.
//  * Both products run on the codes as stored (tcgen05 kind::f8f6f4), keys or
//    value columns in the MMA's 128 rows and the query rows in its N = 2 C
//    columns, which hold two e4m3 terms of each row's operand, 8 rows' first
//    terms, then their second ones:
//      S^T[key, row] = K Q^T, q 2^s = hi + lo (s puts the row's largest near
//        448): exact for components down to 2^-9 of it, as q has 8
//        significant bits and hi leaves at most 4;
//      O^T[d, row] = V^T P^T, P = 2^(x - m') v_scale / R = hi + lo / 16, R the
//        larger v_scale of the tile's two blocks: 8 significant bits where P >=
//        2^-6, below that multiples of 2^-13 (2^-17 of the largest weight or
//        less), rounded with a dither that differs between a tile's 128 keys,
//        so that many equal small weights keep their sum: within 2^-13 a tile.
//  * Softmax: thread = key, 8 or 16 rows; the block's K scale folds into the
//    logit.  m' is a running reference per row that is set by the row's first
//    tile (to put its maximum at 2^4.25) and afterwards only when a weight
//    exceeds 2^8.75, so a tile usually costs one vote of the warps instead of a
//    maximum per row.
//  * A segment's key tiles are taken from the last down: the nearest keys often
//    weigh most (with distance biases always), so m' settles at once.
//  * O^T of each tile is read from tensor memory and added, times R, to sums in
//    registers: no rescaling pass, any scales.
//  * The key tiles of the whole call form one sequence (smla_paged.cuh) that
//    the persistent CTAs share equally, whatever the lengths; a unit that
//    several CTAs share is merged by a second kernel.  Lengths are read on the
//    device only.
//  * Roles: TMA producer, QK^T issuer, P.V issuer, scheduler (segments ahead,
//    their Q split and columns), 4 softmax warps, 4 warps that sum O.
//
// Measured, all launches of a call, D = 128 unless stated, shares of the copy
// bandwidth 6.79 TB/s: 64 requests of up to 16 000 tokens, 8 K/V heads, G = 8
// (1.14 GB) 176 us, 0.95; 3 of up to 260 000, 4 heads, G = 7, distance biases (0.56
// GB) 95 us, 0.87; 200 of up to 500, 8 heads, G = 8 (0.13 GB) 54 us, 0.34: a segment's
// start and end take what 4 of its tiles do; 100 windows of 4096, 5 tokens each, 5
// heads, G = 3, D = 64, capped (0.23 GB) 86 us, 0.39: the chain S, softmax, P V of a
// 16 KB tile takes 1.7 us and one tile per CTA is in its softmax at a time.
#include "smla_paged.cuh"

namespace smla {

namespace {

// Two weights -> e4m3 codes hi and lo of p ~ hi + lo / 16 (low byte from x0).
// The split runs in f16x2: 11 bits, more than the two terms keep.  `dither`, f16x2,
// is added to 16 lo: a thread's share of the steps in which lo counts small weights.
__device__ __forceinline__ void split_p(float x0, float x1, uint32_t dither, uint32_t& hi, uint32_t& lo) {
  uint32_t a, d, r;
  uint16_t t;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(a) : "f"(x1), "f"(x0));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(t) : "r"(a));
  hi = t;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(t));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(d));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(r), "r"(0x4c004c00u), "r"(dither));  // 16, 16
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(t) : "r"(r));
  lo = t;
}
// What a row needs of its own.
template <int C>
struct Columns {
  float scale[C];  // logit = S * scale * k_scale, in log2 units (in caps with softcap)
  float slope[C];  // log2 units per key of distance
  int pos[C], lo[C], hi[C];
};

template <int D, int C>
struct Lay {
  static constexpr int N = 2 * C;          // MMA columns: two terms of each row
  static constexpr int kWarps = 12;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPerSm = 2;
  static constexpr int kKTile = kKeyTile * D;
  static constexpr int kStage = 2 * kKTile;
  static constexpr int kStages = 3 * (128 / D);
  static constexpr int kMeta = 8;          // ring of block scales and flags
  static constexpr int kQBuf = N * D;
  static constexpr int kSegs = 4, kQs = 2;  // segments ahead; their Q and columns
  static constexpr int kPBuf = kKeyTile * N;
  static constexpr int kPBufs = C == 16 ? 1 : 2;   // two where two CTAs still fit an SM
  static constexpr int kRefs = 4;                  // ring of (factors, v scales) towards the summing warps
  static constexpr int kOffQ = kStages * kStage;
  static constexpr int kOffP = kOffQ + kQs * kQBuf;
  static constexpr int kOffCols = kOffP + kPBufs * kPBuf;
  static constexpr int kOffMeta = kOffCols + kQs * (int)sizeof(Columns<C>);
  static constexpr int kOffRefs = kOffMeta + kMeta * 32;
  static constexpr int kRef = C * 4 + 16;          // factor[C], R, whether a factor is not 1
  static constexpr int kOffRed = kOffRefs + kRefs * kRef;          // float [4][C] maxima
  static constexpr int kOffSum = kOffRed + 4 * C * 4;              // float [4][C] sums
  static constexpr int kOffM = kOffSum + 4 * C * 4;                // float [C] m'
  static constexpr int kOffFin = kOffM + C * 4;                    // float [segments][m' | l][C]
  static constexpr int kOffSeg = kOffFin + kSegs * 2 * C * 4;
  static constexpr int kOffBar = (kOffSeg + kSegs * (int)sizeof(Segment) + 7) / 8 * 8;
  enum {
    kKFull = 0, kVFull = kKFull + kStages, kEmpty = kVFull + kStages, kSFull = kEmpty + kStages, kSFree = kSFull + 2,
    kPFull = kSFree + 2, kPFree = kPFull + kPBufs, kOFull = kPFree + kPBufs, kOFree = kOFull + 2,
    kRefFull = kOFree + 2, kSegFull = kRefFull + kRefs, kSegFree = kSegFull + kSegs, kQFull = kSegFree + kSegs,
    kQFree = kQFull + kQs, kFinFull = kQFree + kQs, kDrainQk = kFinFull + kSegs, kDrainPv, kNumBars
  };
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmem = kOffMisc + 16 + 1024;
  static constexpr int kTmemS = 0, kTmemO = 2 * N;  // S [2][N], O [2][N]
  static constexpr int kTmemCols = 4 * N;
  static_assert(kTmemCols >= 32 && kPerSm * kTmemCols <= 512, "tensor memory");
  static_assert(kPerSm * (kSmem + 1024) <= 233472, "shared memory of an SM");
  static_assert(kStage % 1024 == 0 && kQBuf % 1024 == 0 && kOffP % 128 == 0 && kOffCols % 16 == 0 &&
                kOffRefs % 16 == 0 && kRef % 16 == 0 && kOffFin % 16 == 0 && kOffRed % 16 == 0, "alignment");
  static_assert((kMaxPagedRequests + 1 + kWarps) * 8 <= kStages * kStage, "prefix sums fit the stages");
};

// kCap: may have a softcap.
template <int D, int C, bool kCap>
__global__ void __launch_bounds__(Lay<D, C>::kThreads, Lay<D, C>::kPerSm)
    paged_attn_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map) {
  using L = Lay<D, C>;
  constexpr int N = L::N;
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
      mbar_init(&bars[L::kKFull + i], 2);  // the copies, the block's scales
      mbar_init(&bars[L::kVFull + i], 1);
      mbar_init(&bars[L::kEmpty + i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[L::kSFull + i], 1);
      mbar_init(&bars[L::kSFree + i], 4);
      mbar_init(&bars[L::kOFull + i], 1);
      mbar_init(&bars[L::kOFree + i], 4);
      mbar_init(&bars[L::kQFull + i], 1);
      mbar_init(&bars[L::kQFree + i], 1 + 4);
    }
    for (int i = 0; i < L::kPBufs; ++i) {
      mbar_init(&bars[L::kPFull + i], 4);
      mbar_init(&bars[L::kPFree + i], 1);
    }
    for (int i = 0; i < L::kRefs; ++i) mbar_init(&bars[L::kRefFull + i], 1);
    for (int i = 0; i < L::kSegs; ++i) {
      mbar_init(&bars[L::kSegFull + i], 1);
      mbar_init(&bars[L::kSegFree + i], 3 + 4 + 4);
      mbar_init(&bars[L::kFinFull + i], 1);
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
  grid_dependency_wait();  // everything above may overlap the preceding kernel's end
  const PagedRange range = paged_range<L::kThreads>(p, reinterpret_cast<int64_t*>(smem), 2);
  fence_proxy_async_smem();  // the copies may overwrite the prefix sums
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
#define PA_WAIT(idx, parity) wait_bar(&bars[(idx)], (parity), abort_flag, p.status)

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    Ring<L::kStages> ring;
    const int outside = (int)(a.NB * a.HK * kBlock);  // a row behind the cache: reads as zeros
    int tl = 0, seg = 0;
    bool dead = false;
    while (true) {
      const int sb = seg % L::kSegs;
      dead = __any_sync(kAll, !PA_WAIT(L::kSegFull + sb, (seg / L::kSegs) & 1));
      if (dead) break;
      const Segment s = *reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment));
      if (s.n == 0) break;
      const int32_t* row = a.block_table + (int64_t)s.r * a.MB;
      // lane l holds block base - l of the row (tiles are taken from the last down): its cache block (-1: none)
      // and scales; the next 32 are fetched while these are in use
      auto fetch = [&](int page, int& b, float& ks, float& vs) {
        b = -1;
        ks = vs = 0.f;
        if (page >= 0 && page * kBlock < s.hi && (page + 1) * kBlock > s.lo) {
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
      fetch(2 * (s.kt + s.n - 1) + 1 - lane, b, ks, vs);
      for (int i = 0; i < s.n && !dead; ++i, ++tl) {
        const int at = (2 * i) & 31;
        if (at == 0) {
          if (i > 0) {
            b = nb;
            ks = nks;
            vs = nvs;
          }
          if (i + 16 < s.n) fetch(2 * (s.kt + s.n - 1 - i - 16) + 1 - lane, nb, nks, nvs);
        }
        const int b0 = __shfl_sync(kAll, b, at + 1), b1 = __shfl_sync(kAll, b, at);
        const int st = ring.i;
        dead = __any_sync(kAll, !PA_WAIT(L::kEmpty + st, ring.phase ^ 1u));  // (true at once in the first lap)
        if (dead) break;
        ring.next();
        if (lane == 0) {
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
        // the scales arrive while the copies are under way
        const float k0 = __shfl_sync(kAll, ks, at + 1), k1 = __shfl_sync(kAll, ks, at);
        const float v0 = __shfl_sync(kAll, vs, at + 1), v1 = __shfl_sync(kAll, vs, at);
        if (lane == 0) {
          float* meta = reinterpret_cast<float*>(smem + L::kOffMeta + (tl % L::kMeta) * 32);
          *reinterpret_cast<float4*>(meta) = make_float4(k0, k1, v0, v1);
          reinterpret_cast<int*>(meta)[4] = (b0 >= 0 ? 1 : 0) | (b1 >= 0 ? 2 : 0);
          mbar_arrive(&bars[L::kKFull + st]);
        }
        __syncwarp();
      }
      if (dead) break;
      if (lane == 0) mbar_arrive(&bars[L::kSegFree + sb]);
      ++seg;
    }
    // no copy may still be landing when the CTA exits
    for (int j = max(0, tl - L::kStages); j < tl; ++j) {
      mbar_wait_drain(&bars[L::kKFull + j % L::kStages], (j / L::kStages) & 1);
      mbar_wait_drain(&bars[L::kVFull + j % L::kStages], (j / L::kStages) & 1);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- QK^T issuer
    if (lane == 0) {
      constexpr uint32_t id = idesc_e4m3(128, N, 0, 0);
      constexpr uint32_t lay = D == 128 ? kLayoutSw128 : kLayoutSw64;
      const uint64_t dk0 = make_sdesc(smem_u32(smem), 16, 8 * D, lay);
      const uint64_t dq0 = make_sdesc(smem_u32(smem + L::kOffQ), 16, 8 * D, lay);
      Ring<L::kStages> ring;
      int tl = 0, seg = 0;
      bool dead = false;
      while (!dead) {
        const int sb = seg % L::kSegs, qb = seg % L::kQs;
        if (!PA_WAIT(L::kQFull + qb, (seg / L::kQs) & 1)) break;
        const int n = reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment))->n;
        if (n == 0) break;
        mbar_arrive(&bars[L::kSegFree + sb]);
        const uint64_t dq = dq0 + (uint64_t)((qb * L::kQBuf) >> 4);
        for (int i = 0; i < n; ++i, ++tl) {
          const int st = ring.i, buf = tl & 1;
          if (!PA_WAIT(L::kSFree + buf, ((tl >> 1) + 1) & 1) || !PA_WAIT(L::kKFull + st, ring.phase)) {
            dead = true;
            break;
          }
          ring.next();
          tc_fence_after();
          const uint64_t dk = dk0 + (uint64_t)((st * L::kStage) >> 4);
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            mma_f8(tmem + L::kTmemS + buf * N, dk + ((32 * k) >> 4), dq + ((32 * k) >> 4), id, k > 0 ? 1u : 0u);
          mma_commit(&bars[L::kSFull + buf]);
        }
        if (!dead) mma_commit(&bars[L::kQFree + qb]);  // the segment's Q has been read
        ++seg;
      }
      // every issued operation completes before tensor memory is released
      mma_commit(&bars[L::kDrainQk]);
      mbar_wait_drain(&bars[L::kDrainQk], 0);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---------------------------------------------------------------- P.V issuer
    if (lane == 0) {
      constexpr uint32_t id = idesc_e4m3(128, N, 1, 1);
      // V: rows are keys, D-byte swizzle, read MN-major; at D = 64 the MMA's upper 64 rows read the same
      // columns again (atoms 0 bytes apart) and their results are not used
      const uint64_t dv0 = make_sdesc(smem_u32(smem + L::kKTile), 0, 8 * D, D == 128 ? kLayoutSw128 : kLayoutSw64);
      // P: core matrices of 8 keys x 16 columns, the N / 16 of 8 keys together
      const uint64_t dp0 = make_sdesc(smem_u32(smem + L::kOffP), 8 * N, 128, kLayoutNone);
      Ring<L::kStages> ring;
      int tl = 0, seg = 0, left = 0;
      for (;; ++tl, --left) {
        if (left == 0) {  // the next segment's tiles
          const int sb = seg % L::kSegs;
          if (!PA_WAIT(L::kSegFull + sb, (seg / L::kSegs) & 1)) break;
          left = reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment))->n;
          if (left == 0) break;
          mbar_arrive(&bars[L::kSegFree + sb]);
          ++seg;
        }
        const int st = ring.i, buf = tl & 1;
        const int pb = tl % L::kPBufs;
        if (!PA_WAIT(L::kPFull + pb, (tl / L::kPBufs) & 1) || !PA_WAIT(L::kVFull + st, ring.phase) ||
            !PA_WAIT(L::kOFree + buf, ((tl >> 1) + 1) & 1))
          break;
        ring.next();
        tc_fence_after();
        const uint64_t dv = dv0 + (uint64_t)((st * L::kStage) >> 4), dp = dp0 + (uint64_t)((pb * L::kPBuf) >> 4);
#pragma unroll
        for (int step = 0; step < 4; ++step)  // 32 keys
          mma_f8(tmem + L::kTmemO + buf * N, dv + ((32 * D * step) >> 4), dp + ((32 * N * step) >> 4), id,
                 step > 0 ? 1u : 0u);
        mma_commit(&bars[L::kPFree + pb]);
        mma_commit(&bars[L::kEmpty + st]);  // the tile's QK^T completed before its P was written
        mma_commit(&bars[L::kOFull + buf]);
      }
      mma_commit(&bars[L::kDrainPv]);
      mbar_wait_drain(&bars[L::kDrainPv], 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------------------------------------------------------- scheduler
    // For each segment: the record, the rows' columns and the two terms of Q.
    int seg = 0;
    bool dead = false;
    const PagedMerge mine = walk_segments(p, range, [&](const Segment& s, const PagedRequest& q) {
      // what the rows need is under way before the waits: D / 8 lanes per row, 8 values of q each
      constexpr int kLanes = D / 8, kRowsPer = 32 / kLanes;
      const int rows = s.ntok * s.heads, sub = lane / kLanes, c = lane % kLanes;
      const int tok = lane < rows ? lane / s.heads : 0, head = lane < rows ? lane - tok * s.heads : 0;  // of row `lane`
      constexpr int kSteps = C / kRowsPer, kAhead = kSteps < 2 ? kSteps : 2;
      uint4 v[kAhead];
      auto fetch = [&](int step) {  // steps step .. step + kAhead - 1
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int row = (step + i) * kRowsPer + sub;
          const int tr = __shfl_sync(kAll, tok, row), hr = __shfl_sync(kAll, head, row);
          v[i] = make_uint4(0u, 0u, 0u, 0u);
          if (row < rows)
            v[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                        (int64_t)(s.t0 + tr) * a.q_stride + (int64_t)(s.h0 + hr) * D) + c);
        }
      };
      fetch(0);
      const int t = s.t0 + tok, lo = lane < rows ? q.lo(a, t) : 0, hi = lane < rows ? q.hi(t) : 0;
      const float slope = a.alibi_slopes && lane < rows ? __ldg(a.alibi_slopes + s.h0 + head) * kLog2e : 0.f;
      const int sb = seg % L::kSegs, qb = seg % L::kQs;
      if (seg >= L::kSegs) dead = __any_sync(kAll, !PA_WAIT(L::kSegFree + sb, (seg / L::kSegs + 1) & 1));
      if (dead) return false;
      if (lane == 0) {
        *reinterpret_cast<Segment*>(smem + L::kOffSeg + sb * sizeof(Segment)) = s;
        mbar_arrive(&bars[L::kSegFull + sb]);  // the copies may begin
      }
      if (seg >= L::kQs) dead = __any_sync(kAll, !PA_WAIT(L::kQFree + qb, (seg / L::kQs + 1) & 1));
      if (dead) return false;
      Columns<C>* cols = reinterpret_cast<Columns<C>*>(smem + L::kOffCols + qb * sizeof(Columns<C>));
      if (lane < C) {
        cols->pos[lane] = q.pos(t);
        cols->lo[lane] = lo;
        cols->hi[lane] = hi;
        cols->slope[lane] = slope;
      }
      const uint32_t qd = smem_u32(smem + L::kOffQ + qb * L::kQBuf);
#pragma unroll 1
      for (int step = 0; step < kSteps; step += kAhead) {
        if (step > 0) fetch(step);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int row = (step + i) * kRowsPer + sub;
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          uint32_t top = max_u16x2(max_u16x2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                   max_u16x2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) top = max_u16x2(top, __shfl_xor_sync(kAll, top, o));
          const uint32_t amax = max(top << 16, top & 0xffff0000u);  // the largest magnitude's bits
          uint32_t h[2], l[2];
          float back;
          split_q8(w, amax, h, l, back);
          const int op = (row & ~7) + row;  // operand row: 16 b + row % 8, and the second term 8 behind
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(qd + swz<D>(op, c >> 1) + 8 * (c & 1)), "r"(h[0]), "r"(h[1])
                       : "memory");
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(qd + swz<D>(op + 8, c >> 1) + 8 * (c & 1)), "r"(l[0]),
                       "r"(l[1])
                       : "memory");
          if (c == 0) cols->scale[row] = a.sm_scale * back * (kCap && a.softcap > 0.f ? 1.f / a.softcap : kLog2e);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[L::kQFull + qb]);
      ++seg;
      return true;
    });
    if (lane == 0) p.merge[blockIdx.x] = mine;
    const int sb = seg % L::kSegs, qb = seg % L::kQs;
    if (!dead && seg >= L::kSegs) dead = __any_sync(kAll, !PA_WAIT(L::kSegFree + sb, (seg / L::kSegs + 1) & 1));
    if (!dead && seg >= L::kQs) dead = __any_sync(kAll, !PA_WAIT(L::kQFree + qb, (seg / L::kQs + 1) & 1));
    if (lane == 0 && !dead) {
      reinterpret_cast<Segment*>(smem + L::kOffSeg + sb * sizeof(Segment))->n = 0;
      mbar_arrive(&bars[L::kSegFull + sb]);
      mbar_arrive(&bars[L::kQFull + qb]);
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax: thread = key, C rows
    const int quarter = warp & 3;
    const int key = 32 * quarter + lane;
    // (2 k + 1 - 128) 2^-17, k the key's bits in reverse: evenly over half a step of lo to either side
    const float dither_f = (float)(2 * (int)(__brev((uint32_t)key) >> 25) - 127) * 0x1p-17f;
    const uint32_t dither = pack_f16x2(dither_f, dither_f);
    const uint32_t s_addr = tmem + ((uint32_t)(32 * quarter) << 16) + L::kTmemS;
    const uint32_t p_addr = smem_u32(smem + L::kOffP) + (key >> 3) * 8 * N + (key & 7) * 16;
    float* red = reinterpret_cast<float*>(smem + L::kOffRed);
    float* sums = reinterpret_cast<float*>(smem + L::kOffSum);
    float* m_ref = reinterpret_cast<float*>(smem + L::kOffM);
    constexpr int bar = 1;
    constexpr uint32_t kAllSeen = (1u << C) - 1u;
    Ring<L::kStages> ring;
    int tl = 0, seg = 0;
    bool dead = false;
    // `dead` stays the same in the whole warp.  After a wait that ran out the loops go on without waiting to
    // the end of the segment, where the threads of a barrier leave together: none is left behind at one.
    auto wait = [&](int idx, uint32_t parity) {
      const bool ok = !dead && PA_WAIT(idx, parity);
      dead = !__all_sync(kAll, ok);
    };
    while (true) {
      const int sb = seg % L::kSegs, qb = seg % L::kQs;
      wait(L::kQFull + qb, (seg / L::kQs) & 1);
      if (quarter == 0 && lane < C) m_ref[lane] = 0.f;
      dead = bar_any(bar, 128, dead);
      if (dead) break;
      const Segment* sp = reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment));
      const Columns<C>* cols = reinterpret_cast<const Columns<C>*>(smem + L::kOffCols + qb * sizeof(Columns<C>));
      const int kt = sp->kt, n = sp->n;
      if (n == 0) break;
      uint32_t seen = 0u;  // rows that have met a key they see (the same in every thread of the group)
      uint64_t l2[C / 2];
#pragma unroll
      for (int c = 0; c < C / 2; ++c) l2[c] = 0ull;
      for (int i = n - 1; i >= 0; --i, ++tl, ring.next()) {
        const int buf = tl & 1, st = ring.i, pb = tl % L::kPBufs;
        {
          // the tile's scales and flags (behind its K copies), and its S
          const bool ok = !dead && PA_WAIT(L::kKFull + st, ring.phase) && PA_WAIT(L::kSFull + buf, (tl >> 1) & 1);
          dead = !__all_sync(kAll, ok);
        }
        tc_fence_after();
        const float* meta = reinterpret_cast<const float*>(smem + L::kOffMeta + (tl % L::kMeta) * 32);
        const float ks = meta[key >> 6], ref_v = fmaxf(fabsf(meta[2]), fabsf(meta[3]));
        const float vf = ref_v > 0.f ? __fdividef(meta[2 + (key >> 6)], ref_v) : 0.f;
        const int pages = reinterpret_cast<const int*>(meta)[4];
        const int j0 = (kt + i) * kKeyTile, j = j0 + key;
        float y[C];  // logits, then logits - m'
        {
          const uint64_t ks2 = pack2(ks, ks);
#pragma unroll
          for (int b = 0; b < C / 8; ++b) {
            uint32_t raw[16];
            tmem_ld16_sync(s_addr + buf * N + 16 * b, raw);
#pragma unroll
            for (int c = 0; c < 8; c += 2) {
              const float2 f = *reinterpret_cast<const float2*>(&cols->scale[8 * b + c]);
              const float2 v = unpack2(mul2(add2(pack2(__uint_as_float(raw[c]), __uint_as_float(raw[c + 1])),
                                                 pack2(__uint_as_float(raw[8 + c]), __uint_as_float(raw[9 + c]))),
                                            mul2(pack2(f.x, f.y), ks2)));
              y[8 * b + c] = v.x;
              y[8 * b + c + 1] = v.y;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kSFree + buf]);
        if (kCap && a.softcap > 0.f) {
          // y is x / cap.  The polynomial alone where it holds for all, else each by its own size.
          const float cap = a.softcap * kLog2e;
          float most = 0.f;
#pragma unroll
          for (int c = 0; c < C; ++c) most = fmaxf(most, fabsf(y[c]));
          if (__all_sync(kAll, most * most <= kTanhTop)) {
#pragma unroll
            for (int c = 0; c < C; c += 2) {
              const uint64_t u = pack2(y[c], y[c + 1]), u2 = mul2(u, u);
              uint64_t t = pack2(cap * kTanh[4], cap * kTanh[4]);
#pragma unroll
              for (int d = 3; d >= 0; --d) t = fma2(t, u2, pack2(cap * kTanh[d], cap * kTanh[d]));
              const float2 v = unpack2(mul2(u, t));
              y[c] = v.x;
              y[c + 1] = v.y;
            }
          } else {
#pragma unroll
            for (int c = 0; c < C; ++c) y[c] = cap * tanh_any(y[c]);
          }
        }
        if (a.alibi_slopes) {
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&cols->slope[c]);
            const int4 at = *reinterpret_cast<const int4*>(&cols->pos[c]);
            y[c] = fmaf(-f.x, (float)abs(at.x - j), y[c]);
            y[c + 1] = fmaf(-f.y, (float)abs(at.y - j), y[c + 1]);
            y[c + 2] = fmaf(-f.z, (float)abs(at.z - j), y[c + 2]);
            y[c + 3] = fmaf(-f.w, (float)abs(at.w - j), y[c + 3]);
          }
        }
        const bool inside = j0 >= sp->all_lo && j0 + kKeyTile <= sp->all_hi && pages == 3;  // every row sees every key
        bool zero_v = false;
        if (!inside) {
          const bool page_ok = (pages >> (key >> 6)) & 1;
#pragma unroll
          for (int c = 0; c < C; ++c)  // (no branches)
            y[c] = page_ok & (j >= cols->lo[c]) & (j < cols->hi[c]) ? y[c] : -INFINITY;
          // keys that no row sees may hold any codes: their V rows become zeros
          zero_v = j < sp->lo || j >= sp->hi;
          if (__any_sync(kAll, zero_v)) wait(L::kVFull + st, ring.phase);
        }
        float over = -INFINITY;
#pragma unroll
        for (int c = 0; c < C; c += 4) {
          const float4 m = *reinterpret_cast<const float4*>(&m_ref[c]);
          y[c] -= m.x;
          y[c + 1] -= m.y;
          y[c + 2] -= m.z;
          y[c + 3] -= m.w;
          over = fmaxf(over, fmaxf(fmaxf(y[c], y[c + 1]), fmaxf(y[c + 2], y[c + 3])));
        }
        const bool refresh = bar_any(bar, 128, over > kTop) || seen != kAllSeen;
        // the factors go to the summing warps: slot tl % 4 was read before P.V of tile tl - 2 could be issued
        uint8_t* ref = smem + L::kOffRefs + (tl % L::kRefs) * L::kRef;
        wait(L::kPFree + pb, (tl / L::kPBufs + 1) & 1);  // P.V has read this P buffer
        if (refresh) {
          // lane c (mod C): row c's maximum, the change of its reference, and the factor of its sums
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const float v = warp_max(y[c]);
            if ((lane & (C - 1)) == c) mx = v;
          }
          if (lane < C) red[quarter * C + lane] = mx;
          named_bar_sync(bar, 128);
          const int c1 = lane & (C - 1);
          mx = fmaxf(fmaxf(red[c1], red[C + c1]), fmaxf(red[2 * C + c1], red[3 * C + c1]));
          const bool first = !((seen >> c1) & 1u);
          const bool set = first ? mx > -INFINITY : mx > kTop;
          const float up = set ? mx - kRefresh : 0.f, factor = set && !first ? ex2_approx(-up) : 1.f;
          seen |= __ballot_sync(kAll, set) & kAllSeen;
          if (quarter == 0 && lane < C) {
            m_ref[lane] += up;
            reinterpret_cast<float*>(ref)[lane] = factor;
          }
#pragma unroll
          for (int c = 0; c < C; c += 2) {
            y[c] -= __shfl_sync(kAll, up, c);
            y[c + 1] -= __shfl_sync(kAll, up, c + 1);
            l2[c / 2] = mul2(l2[c / 2], pack2(__shfl_sync(kAll, factor, c), __shfl_sync(kAll, factor, c + 1)));
          }
          named_bar_sync(bar, 128);  // m_ref and red are in order for the next tile
        }
        if (quarter == 0 && lane == 0) {
          reinterpret_cast<float*>(ref)[C] = ref_v;
          reinterpret_cast<int*>(ref)[C + 1] = refresh;
        }
        const uint64_t vf2 = pack2(vf, vf);
#pragma unroll
        for (int b = 0; b < C / 8; ++b) {
          uint32_t hw[4], lw[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int at = 8 * b + 2 * c;
            const uint64_t p2 = pack2(ex2_approx(y[at]), ex2_approx(y[at + 1]));
            l2[at / 2] = add2(l2[at / 2], p2);
            const float2 pv = unpack2(mul2(p2, vf2));
            split_p(pv.x, pv.y, dither, hw[c], lw[c]);
          }
          st_shared_v4(p_addr + pb * L::kPBuf + 128 * b, hw[0] | (hw[1] << 16), hw[2] | (hw[3] << 16),
                       lw[0] | (lw[1] << 16), lw[2] | (lw[3] << 16));
        }
        if (zero_v) {
          const uint32_t v = smem_u32(smem + st * L::kStage + L::kKTile) + key * D;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) st_shared_v4(v + 16 * k, 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars[L::kPFull + pb]);
          if (quarter == 0) mbar_arrive(&bars[L::kRefFull + tl % L::kRefs]);
        }
      }
      // the rows' sums over the segment's keys
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float2 pair = unpack2(l2[c / 2]);
        float v = c & 1 ? pair.y : pair.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
        if (lane == c) sums[quarter * C + c] = v;
      }
      named_bar_sync(bar, 128);
      if (quarter == 0) {
        float* fin = reinterpret_cast<float*>(smem + L::kOffFin + sb * 2 * C * 4);
        if (lane < C) {
          const float l = (sums[lane] + sums[C + lane]) + (sums[2 * C + lane] + sums[3 * C + lane]);
          fin[lane] = l == 0.f ? kNoMax : m_ref[lane];
          fin[C + lane] = l;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kFinFull + sb]);
      }
      if (lane == 0) {
        mbar_arrive(&bars[L::kQFree + qb]);
        mbar_arrive(&bars[L::kSegFree + sb]);
      }
      ++seg;
    }
  } else {
    // ---------------------------------------------------------------- sums of O: thread = value column, C rows
    const int quarter = warp & 3, d = 32 * quarter + lane;
    const uint32_t o_addr = tmem + ((uint32_t)(32 * quarter) << 16) + L::kTmemO;
    int tl = 0, seg = 0;
    bool dead = false;
    auto wait = [&](int idx, uint32_t parity) {
      const bool ok = !dead && PA_WAIT(idx, parity);
      dead = !__all_sync(kAll, ok);
    };
    while (true) {
      const int sb = seg % L::kSegs;
      wait(L::kSegFull + sb, (seg / L::kSegs) & 1);
      if (dead) break;
      const Segment* sp = reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment));
      const int n = sp->n;
      if (n == 0) break;
      float acc[C];
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] = 0.f;
      for (int i = 0; i < n; ++i, ++tl) {
        const int buf = tl & 1;
        wait(L::kRefFull + tl % L::kRefs, (tl / L::kRefs) & 1);
        const uint8_t* ref = smem + L::kOffRefs + (tl % L::kRefs) * L::kRef;
        const float ref_v = reinterpret_cast<const float*>(ref)[C];
        if (reinterpret_cast<const int*>(ref)[C + 1]) {
#pragma unroll
          for (int c = 0; c < C; ++c) acc[c] *= reinterpret_cast<const float*>(ref)[c];
        }
        wait(L::kOFull + buf, (tl >> 1) & 1);
        if (dead) break;
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < C / 8; ++b) {
          uint32_t o[16];
          tmem_ld16_sync(o_addr + buf * N + 16 * b, o);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            acc[8 * b + c] =
                fmaf(fmaf(__uint_as_float(o[8 + c]), 1.f / 16.f, __uint_as_float(o[c])), ref_v, acc[8 * b + c]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kOFree + buf]);
      }
      wait(L::kFinFull + sb, (seg / L::kSegs) & 1);
      if (dead) break;
      const float* fin = reinterpret_cast<const float*>(smem + L::kOffFin + sb * 2 * C * 4);
      const int heads = sp->heads, rows = sp->ntok * heads;
      if (sp->slot < 0) {
        // lane c: row c's place and 1 / l
        const int64_t first = (int64_t)sp->t0 * a.H + sp->h0;
        const float l = lane < C ? fin[C + lane] : 0.f, inv = l == 0.f ? 0.f : 1.f / l;
        const int at = lane / heads * a.H + lane % heads;
        if (quarter == 0 && lane < rows) a.lse[first + at] = l == 0.f ? -INFINITY : (fin[lane] + log2f(l)) * kLn2;
        if (32 * quarter < D) {
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + first * D + d;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int64_t to = __shfl_sync(kAll, at, c);
            const float f = __shfl_sync(kAll, inv, c);
            if (c < rows) out[to * D] = __float2bfloat16(acc[c] * f);
          }
        }
      } else {
        const int64_t part = 2 * (int64_t)blockIdx.x + sp->slot;
        float* o = p.part_o + part * C * D;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (c >= rows) break;
          if (D == 128 || d < D) o[c * D + d] = acc[c];
        }
        if (d < 2 * C) p.part_ml[part * 2 * C + d] = fin[d];
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

// Places of a unit beside its tiles: about what its start and end take (32 requests of 5 tokens, G = 4: 2, 3, 4,
// 6, 8 give 77.0, 76.5, 75.5, 75.7, 77.0 us).
constexpr int kUnitCost = 4;

template <int D, int C>
cudaError_t launch(const PagedAttnArgs& a, int num_sms, cudaStream_t stream) {
  using L = Lay<D, C>;
  CUtensorMap k_map, v_map;
  cudaError_t e = cache_maps(a, &k_map, &v_map);
  if (e != cudaSuccess) return e;
  const PagedParams p = paged_params<C>(a, paged_sizes(C, D, L::kPerSm, num_sms), kUnitCost);
  // 16 rows: a kernel without the cap's code where there is none (32 requests of 5 tokens, G = 4: 76.9 us, 81.5 with
  // it); 8 rows: one for both (64 long requests 175 us, with two of its registers spilled 178).
  e = launch_overlapped(C == 8 || a.softcap > 0.f ? paged_attn_kernel<D, C, true> : paged_attn_kernel<D, C, C == 8>,
                        dim3((unsigned)p.ctas), L::kThreads, L::kSmem, stream, p, k_map, v_map);
  return e == cudaSuccess ? launch_merge<D, C>(p, stream) : e;
}

// Rows per query tile, by those of a request and K/V head (its heads times the estimated tokens).  Fewer
// rows cost less softmax work per key, more let a key read once meet them all; tiles of 256 rows take the
// same for few as for many.  128 requests of up to 8000 tokens, 4 K/V heads, D = 128 (300 of up to 2000, 8 K/V
// heads), tiles of 8 | 16 | 256: 16 rows 133 (185) | 112 (206) | 231 (300) us; 32 rows 205 (310) | 149 (302) | 232
// (306); 48 rows 272 (442) | 187 (417) | 234 (311); 64 rows 357 (543) | 241 (504) | 236 (321).
int rows_for(int G, int max_query_len) {
  const int64_t rows = (int64_t)G * std::max(1, max_query_len);
  return rows <= 8 ? 8 : rows <= 48 ? 16 : 256;
}

}  // namespace

size_t paged_attention_workspace(int T, int H, int HK, int D, int R, int max_query_len, int num_sms) {
  const int C = rows_for(H / HK, max_query_len);
  return C == 256 ? paged_prefill_workspace(T, H, D, R, num_sms) : paged_sizes(C, D, 2, num_sms).bytes;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, int max_query_len, int num_sms, cudaStream_t stream) {
  const int C = rows_for(a.H / a.HK, max_query_len);
  if (C == 256) return launch_paged_prefill(a, num_sms, stream);
  if (C == 8) return a.D == 128 ? launch<128, 8>(a, num_sms, stream) : launch<64, 8>(a, num_sms, stream);
  return a.D == 128 ? launch<128, 16>(a, num_sms, stream) : launch<64, 16>(a, num_sms, stream);
}

cudaError_t paged_attn_timed_out(int** word) { return timed_out_word(word); }
cudaError_t paged_attn_wait_check(int* status, cudaStream_t stream) { return wait_check(status, stream); }

}  // namespace smla
