// Attention over the paged 8-bit K/V cache for many rows per K/V head: prompts,
// chunks of them, and many heads per K/V head.  What is computed and how the
// call is cut into segments: smla_paged_attn.cu, smla_paged.cuh.
//
// A query tile has 2 x 128 rows (tokens x heads of one K/V head); each half
// meets every key tile of 128 keys in two products of 128 x 128 x D, so the
// tensor cores bound it, with the softmax and the shared memory that feeds the
// products close behind.  One half's softmax runs under the other's products.
//  * S [row][key] = Q K^T on the codes as stored (kind::f8f6f4), q in two e4m3
//    terms (exact but for components below 2^-9 of their row's largest): two
//    passes at the 8-bit rate cost what one at the 16-bit rate would, without
//    converting K.
//  * O += P V in f16 (kind::f16): P then needs one conversion per pair, where two
//    8-bit terms need five, and V is converted once for the 256 rows.  The
//    conversion also applies v_scale / R (R the largest v_scale of the segment:
//    at most 1) and zeroes the keys that no row sees, whose codes may be
//    anything.  P keeps 11 bits down to 2^-14, below that multiples of 2^-24.
//  * Softmax: thread pair = row, each thread the keys of one block (one K
//    scale).  P = 2^(x - m') with the row's running reference m', computed in one
//    pass over S into registers.  m' starts at 0 and stays there while the row's
//    logits lie where f16 is exact enough; only if a thread's weights add up to
//    65000, a row's first keys to less than 2^-3 or its first 512 to less than 2^4
//    is it refreshed (to put the tile's largest, or in the last case the sum, at
//    2^4), O scaled in tensor memory and the pass repeated.
//  * P overwrites S in tensor memory and enters P V from there.
//  * q is split by a kernel beforehand, so that a segment's Q is one copy that
//    overlaps the end of the segment before.
//  * Masks, caps and slopes change S in tensor memory before the pass, in a loop
//    of their own: unrolled into it they ran out of the instruction caches (three
//    prompts without any: 447 us, then 413).
//  * Roles: TMA producer, MMA issuer, scheduler, 4 warps converting V, 8 softmax
//    warps per half, which also write the results.
//
// Measured, all launches of a call: three prompts of up to 2500 tokens over up
// to 6000 cached ones, 8 K/V heads, G = 4, D = 128 (0.37 TFLOP): 396 us, 0.93 PFLOP/s,
// 0.48 of what a bf16 matrix product reaches; alone the kernel takes 373 us (tensor
// pipe active 44 % of it), the split of q 21, the merge 18.  A half's chain of S (512
// clocks), softmax (1400), P V (512) and four handovers (150 - 300 each) bounds it: S
// and P share their tensor memory, so the next S waits for P V, and two halves
// fill it.  Five prompts of up to 1300 tokens, G = 12, D = 64, capped, packed
// documents: 77 us, bound by short segments (2 tiles) and by the softmax, which with
// cap and masks takes 4200 clocks a tile.
#include "smla_paged.cuh"

namespace smla {

namespace {

constexpr int kRows = 128;          // rows of a half
constexpr float kTop16 = 65000.f;   // largest sum of a thread's weights P = 2^(x - m') (f16: 65504)
constexpr float kRefresh16 = 4.f;   // a refreshed m' puts the tile's maximum (or the row's sum) at 2^4
constexpr float kLow16 = 0x1p-3f;   // a row whose first keys weigh less is refreshed
// A row that weighs less than kThin16 with kThinAt more tiles has its sum put there (the tile's largest weight to 2^9 at
// most): of any later key at most 2^-25 is lost to f16, 2^-29 of the sum, and these add up over long contexts.  Not
// at the first tile, in which the diagonal leaves many rows a few keys.
constexpr float kThin16 = 0x1p4f;
constexpr int kThinAt = 3;
// Places of a unit beside its tiles: about what its start and end take (the prompts above: 1, 2, 3, 4, 6 give 480,
// 412, 412, 415, 420 us; the packed documents 93, 93, 101, 98, 99, before their query tiles were counted by several lanes).
constexpr int kUnitCost = 2;

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int D>
struct PreLay {
  static constexpr int kConvWarp0 = 4, kSoftWarp0 = 8;
  static constexpr int kWarps = 24, kThreads = 32 * kWarps, kPerSm = 1;
  static constexpr int kKTile = kKeyTile * D;               // codes of a tile: K's, V's
  static constexpr int kStages = 3 * (128 / D), kVStages = 2 * (128 / D);
  static constexpr int kV16 = kKeyTile * D * 2;             // converted V: D / 64 panels of 128 keys x 128 bytes
  static constexpr int kMeta = kStages <= 3 ? 8 : 16;       // ring of block scales and flags
  static constexpr int kQTerm = kRows * D, kQHalf = 2 * kQTerm;
  static constexpr int kSegs = 2;
  static constexpr int kOffV = kStages * kKTile;
  static constexpr int kOffV16 = kOffV + kVStages * kKTile;
  static constexpr int kOffQ = kOffV16 + 2 * kV16;
  static constexpr int kOffMeta = kOffQ + 2 * kQHalf;
  static constexpr int kOffRed = kOffMeta + kMeta * 32;            // float [2 halves][2][128] maxima
  static constexpr int kOffSum = kOffRed + 4 * kRows * 4;          // float [2 halves][2][128] sums
  static constexpr int kOffRef = kOffSum + 4 * kRows * 4;          // float [segs] largest v scale
  static constexpr int kOffSeg = kOffRef + 16;
  static constexpr int kOffBar = (kOffSeg + kSegs * (int)sizeof(Segment) + 7) / 8 * 8;
  enum {
    kKFull = 0, kKEmpty = kKFull + kStages, kVFull = kKEmpty + kStages, kVEmpty = kVFull + kVStages,
    kMetaFull = kVEmpty + kVStages, kV16Full = kMetaFull + kMeta, kV16Empty = kV16Full + 2, kSFull = kV16Empty + 2,
    kPFull = kSFull + 2, kPvDone = kPFull + 2, kQFull = kPvDone + 2, kQEmpty = kQFull + 2, kOFree = kQEmpty + 2,
    kSegFull = kOFree + 2,
    kSegFree = kSegFull + kSegs, kDrain = kSegFree + kSegs, kNumBars
  };
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmem = kOffMisc + 16 + 1024;
  static constexpr int kTmemS = 0, kTmemO = 256, kTmemCols = 512;  // S of the halves, O of the halves: 128 columns each
  static_assert(kSmem <= 232448, "shared memory");
  static_assert((kMaxPagedRequests + 1 + kWarps) * 8 <= kOffQ, "prefix sums fit the memory before Q");
  static_assert(kKTile % 1024 == 0 && kV16 % 1024 == 0 && kQTerm % 1024 == 0, "operand alignment");
};

// q in two e4m3 terms per (token, head): q 2^s = hi + lo, s such that the row's
// largest comes near 448.  terms [2][T, H, D]; scale [T, H] = what turns a
// product with K codes into a logit, but for the block's K scale.  D / 8 lanes
// per row, 8 values each; bound by HBM.
constexpr int kSplitThreads = 256;

template <int D>
__global__ void __launch_bounds__(kSplitThreads)
    paged_split_q_kernel(const __grid_constant__ PagedAttnArgs a, uint8_t* __restrict__ terms, float* __restrict__ scale) {
  grid_launch_dependents();
  grid_dependency_wait();
  constexpr int kLanes = D / 8;
  const int64_t rows = (int64_t)a.T * a.H, row0 = (int64_t)clamp_start(a.query_start, 0, a.T) * a.H;
  const int64_t row1 = (int64_t)clamp_start(a.query_start, a.R, a.T) * a.H;
  const int64_t row = ((int64_t)blockIdx.x * kSplitThreads + threadIdx.x) / kLanes;
  const int c = threadIdx.x % kLanes;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  const bool mine = row >= row0 && row < row1;
  if (mine)
    v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + row / a.H * a.q_stride +
                                             row % a.H * D) + c);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t amax = 0u;  // of the magnitudes' bits
#pragma unroll
  for (int k = 0; k < 4; ++k) amax = max(amax, max((w[k] << 16) & 0x7fffffffu, w[k] & 0x7fff0000u));
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) amax = max(amax, __shfl_xor_sync(kAll, amax, o));
  if (!mine) return;
  float back;
  uint32_t hi[2], lo[2];
  split_q8(w, amax, hi, lo, back);
  *reinterpret_cast<uint2*>(terms + row * D + 8 * c) = make_uint2(hi[0], hi[1]);
  *reinterpret_cast<uint2*>(terms + (rows + row) * D + 8 * c) = make_uint2(lo[0], lo[1]);
  if (c == 0) scale[row] = a.sm_scale * back * (a.softcap > 0.f ? 1.f / a.softcap : kLog2e);
}

// First document start of each query tile, a warp each: the shares of the CTAs
// go by the keys that tiles really meet.
__global__ void __launch_bounds__(kSplitThreads)
    paged_tile_doc_kernel(const __grid_constant__ PagedParams p, int32_t* __restrict__ tile_doc, int slots) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int u = ((int)blockIdx.x * kSplitThreads + (int)threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (u >= slots) return;
  const PagedAttnArgs& a = p.a;
  const int r = search_units(a.R, u, [&](int i) { return clamp_start(a.query_start, i, a.T) / p.tq + i; });
  const int t0 = clamp_start(a.query_start, r, a.T), t1 = clamp_start(a.query_start, r + 1, a.T);
  const int64_t ta = t0 + (int64_t)(u - (t0 / p.tq + r)) * p.tq;
  int doc = 0x7fffffff;
  if (ta >= t0)
    for (int64_t t = ta + lane; t < min(ta + p.tq, (int64_t)t1); t += 32) doc = min(doc, __ldg(a.doc_start + t));
  doc = __reduce_min_sync(kAll, doc);
  if (lane == 0) tile_doc[u] = doc;
}

// A 3-D tiled TMA load of one box, as tma_load_2d.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// kBent: with a softcap or slopes.
template <int D, bool kBent>
__global__ void __launch_bounds__(PreLay<D>::kThreads, PreLay<D>::kPerSm)
    paged_prefill_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap q_map) {
  using L = PreLay<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  grid_launch_dependents();  // the merge may be launched behind this grid; it waits for the grid's end
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedAttnArgs& a = p.a;
  const int half_tokens = p.tq / 2;

  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&bars[L::kKFull + i], 1);
      mbar_init(&bars[L::kKEmpty + i], 1);
    }
    for (int i = 0; i < L::kVStages; ++i) {
      mbar_init(&bars[L::kVFull + i], 1);
      mbar_init(&bars[L::kVEmpty + i], 4);
    }
    for (int i = 0; i < L::kMeta; ++i) mbar_init(&bars[L::kMetaFull + i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[L::kV16Full + i], 4);
      mbar_init(&bars[L::kV16Empty + i], 1);
      mbar_init(&bars[L::kSFull + i], 1);
      mbar_init(&bars[L::kPFull + i], 8);
      mbar_init(&bars[L::kPvDone + i], 1);
      mbar_init(&bars[L::kQFull + i], 1);
      mbar_init(&bars[L::kQEmpty + i], 1);
      mbar_init(&bars[L::kOFree + i], 8);
    }
    for (int i = 0; i < L::kSegs; ++i) {
      mbar_init(&bars[L::kSegFull + i], 1);
      mbar_init(&bars[L::kSegFree + i], 2 + 4 + 16);
    }
    mbar_init(&bars[L::kDrain], 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 3) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  // the rows behind a tile's last stay zero: the copies of Q write the rows of its tokens only
  for (int i = tid; i < 2 * L::kQHalf / 16; i += L::kThreads)
    *reinterpret_cast<uint4*>(smem + L::kOffQ + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
  grid_dependency_wait();  // everything above may overlap the preceding kernel's end
  const PagedRange range = paged_range<L::kThreads>(p, reinterpret_cast<int64_t*>(smem), 2);
  fence_proxy_async_smem();  // the copies may overwrite the prefix sums, the tensor cores read the zeros
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
#define PA_WAIT(idx, parity) wait_bar(&bars[(idx)], (parity), abort_flag, p.status)

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    const int outside = (int)(a.NB * a.HK * kBlock);  // a row behind the cache: reads as zeros
    const uint32_t q_bytes = (uint32_t)(p.Gr * half_tokens * D);  // of a half's term
    Ring<L::kStages> ring;
    Ring<L::kVStages> v_ring;
    int tl = 0, seg = 0, filled[2] = {0, 0};
    bool dead = false;
    while (true) {
      const int sb = seg % L::kSegs;
      dead = __any_sync(kAll, !PA_WAIT(L::kSegFull + sb, (seg / L::kSegs) & 1));
      if (dead) break;
      const Segment s = *reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment));
      if (s.n == 0) break;
      const int32_t* row = a.block_table + (int64_t)s.r * a.MB;
      for (int h = 0; h < (s.ntok > half_tokens ? 2 : 1); ++h) {
        if (filled[h] > 0) dead = __any_sync(kAll, !PA_WAIT(L::kQEmpty + h, (filled[h] + 1) & 1));
        if (dead) break;
        ++filled[h];
        if (lane == 0) {
          const uint32_t qd = smem_u32(smem + L::kOffQ + h * L::kQHalf);
          mbar_arrive_expect_tx(&bars[L::kQFull + h], 2 * q_bytes);
          tma_load_3d(qd, &q_map, 0, s.h0, s.t0 + h * half_tokens, &bars[L::kQFull + h]);
          tma_load_3d(qd + L::kQTerm, &q_map, 0, s.h0, a.T + s.t0 + h * half_tokens, &bars[L::kQFull + h]);
        }
        __syncwarp();
      }
      if (dead) break;
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
      for (int i = 0; i < s.n; ++i, ++tl) {
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
        const int st = ring.i, sv = v_ring.i;
        const uint32_t k_phase = ring.phase;
        dead = __any_sync(kAll, !PA_WAIT(L::kKEmpty + st, k_phase ^ 1u));  // (true at once in the first lap)
        if (dead) break;
        const int y0 = b0 >= 0 ? (b0 * a.HK + s.g) * kBlock : outside;
        const int y1 = b1 >= 0 ? (b1 * a.HK + s.g) * kBlock : outside;
        if (lane == 0) {
          const uint32_t kd = smem_u32(smem + st * L::kKTile);
          mbar_arrive_expect_tx(&bars[L::kKFull + st], L::kKTile);
          tma_load_2d(kd, &k_map, 0, y0, &bars[L::kKFull + st]);
          tma_load_2d(kd + kBlock * D, &k_map, 0, y1, &bars[L::kKFull + st]);
        }
        __syncwarp();
        dead = __any_sync(kAll, !PA_WAIT(L::kVEmpty + sv, v_ring.phase ^ 1u));
        if (lane == 0 && !dead) {
          const uint32_t vd = smem_u32(smem + L::kOffV + sv * L::kKTile);
          mbar_arrive_expect_tx(&bars[L::kVFull + sv], L::kKTile);
          tma_load_2d(vd, &v_map, 0, y0, &bars[L::kVFull + sv]);
          tma_load_2d(vd + kBlock * D, &v_map, 0, y1, &bars[L::kVFull + sv]);
        }
        __syncwarp();
        if (dead) {  // this tile's K copies are in flight, its V copies are not
          mbar_wait_drain(&bars[L::kKFull + st], k_phase);
          break;
        }
        // The scales arrive while the copies are under way.  Slot tl % kMeta: its tile before had its S read
        // before its K stage was free again.
        const float k0 = __shfl_sync(kAll, ks, at + 1), k1 = __shfl_sync(kAll, ks, at);
        const float v0 = __shfl_sync(kAll, vs, at + 1), v1 = __shfl_sync(kAll, vs, at);
        if (lane == 0) {
          float* meta = reinterpret_cast<float*>(smem + L::kOffMeta + (tl % L::kMeta) * 32);
          *reinterpret_cast<float4*>(meta) = make_float4(k0, k1, v0, v1);
          reinterpret_cast<int*>(meta)[4] = (b0 >= 0 ? 1 : 0) | (b1 >= 0 ? 2 : 0);
          mbar_arrive(&bars[L::kMetaFull + tl % L::kMeta]);
        }
        __syncwarp();
        ring.next();
        v_ring.next();
      }
      if (dead) break;
      if (lane == 0) mbar_arrive(&bars[L::kSegFree + sb]);
      ++seg;
    }
    // no copy may still be landing when the CTA exits
    for (int h = 0; h < 2; ++h)
      if (filled[h] > 0) mbar_wait_drain(&bars[L::kQFull + h], (filled[h] + 1) & 1);
    for (int j = max(0, tl - L::kStages); j < tl; ++j) mbar_wait_drain(&bars[L::kKFull + j % L::kStages], (j / L::kStages) & 1);
    for (int j = max(0, tl - L::kVStages); j < tl; ++j)
      mbar_wait_drain(&bars[L::kVFull + j % L::kVStages], (j / L::kVStages) & 1);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    // Half h's tile i: S_h = Q_h K_i^T, then, its P written, O_h += P_h V_i and S_h of tile i + 1, which
    // overwrites P and so waits for that product.
    if (lane == 0) {
      constexpr uint32_t id_qk = idesc_e4m3(128, kKeyTile, 0, 0), id_pv = make_idesc_f16(128, D, 0, 1);
      constexpr uint32_t lay = D == 128 ? kLayoutSw128 : kLayoutSw64;
      const uint64_t dk0 = make_sdesc(smem_u32(smem), 16, 8 * D, lay);
      const uint64_t dq0 = make_sdesc(smem_u32(smem + L::kOffQ), 16, 8 * D, lay);
      // converted V, read MN-major: panels of 64 columns
      const uint64_t dv0 = make_sdesc(smem_u32(smem + L::kOffV16), kKeyTile * 128, 1024, kLayoutSw128);
      int tl = 0, seg = 0, done[2] = {0, 0}, filled[2] = {0, 0};  // by half: products P V issued, segments begun
      int was = 0;  // halves of the segment before
      bool dead = false;
      auto wait = [&](int idx, uint32_t parity) {
        if (!dead) dead = !PA_WAIT(idx, parity);
        return !dead;
      };
      Ring<L::kStages> ring;  // the K tile that the next first half takes
      // What a product that is seen to have ended leaves free: P V of half 0 its tile's K (both halves' S came
      // before it), that of the last half its V.  (An arrival here is cheaper than a commit of its own.)
      Ring<L::kStages> k_ring;
      int k_due = 0, v_due = -1;
      auto ended = [&](int h, bool last) {
        if (h == 0 && k_due) {
          mbar_arrive(&bars[L::kKEmpty + k_ring.i]);
          k_ring.next();
          k_due = 0;
        }
        if (last && v_due >= 0) {
          mbar_arrive(&bars[L::kV16Empty + v_due]);
          v_due = -1;
        }
      };
      auto qk = [&](int h, bool last, bool ends) {
        const int st = ring.i;
        if (!wait(L::kKFull + st, ring.phase)) return;
        if (done[h] > 0 && !wait(L::kPvDone + h, (done[h] + 1) & 1)) return;
        ended(h, last);
        tc_fence_after();
        const uint64_t dk = dk0 + (uint64_t)((st * L::kKTile) >> 4), dq = dq0 + (uint64_t)((h * L::kQHalf) >> 4);
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            mma_f8(tmem + L::kTmemS + 128 * h, dq + ((term * L::kQTerm + 32 * k) >> 4), dk + ((32 * k) >> 4), id_qk,
                   term + k > 0 ? 1u : 0u);
        mma_commit(&bars[L::kSFull + h]);
        if (last) ring.next();
        if (ends) mma_commit(&bars[L::kQEmpty + h]);
      };
      auto pv = [&](int h, int t, bool first, bool last) {
        const int vb = t & 1;
        // a segment's first product overwrites O, which the segment before has to have been read out of
        if (first && filled[h] > 1 && !wait(L::kOFree + h, filled[h] & 1)) return;
        if (!wait(L::kPFull + h, done[h] & 1) || !wait(L::kV16Full + vb, (t >> 1) & 1)) return;
        tc_fence_after();
        const uint64_t dv = dv0 + (uint64_t)((vb * L::kV16) >> 4);
#pragma unroll
        for (int k = 0; k < kKeyTile / 16; ++k)  // P: block b's 64 keys in columns 64 b .. 64 b + 31
          mma_ts(tmem + L::kTmemO + 128 * h, tmem + L::kTmemS + 128 * h + 64 * (k >> 2) + 8 * (k & 3),
                 dv + ((2048 * k) >> 4), id_pv, (!first || k > 0) ? 1u : 0u);
        mma_commit(&bars[L::kPvDone + h]);
        if (h == 0) k_due = 1;
        if (last) v_due = vb;
        ++done[h];
      };
      while (true) {
        const int sb = seg % L::kSegs;
        if (!wait(L::kSegFull + sb, (seg / L::kSegs) & 1)) break;
        const Segment* sp = reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment));
        const int n = sp->n, halves = sp->ntok > half_tokens ? 2 : 1;
        if (n == 0) break;
        mbar_arrive(&bars[L::kSegFree + sb]);
        // (the segment before may have had another number of halves)
        if (done[0] > 0 && wait(L::kPvDone, (done[0] + 1) & 1)) ended(0, was == 1);
        if (done[1] > 0 && wait(L::kPvDone + 1, (done[1] + 1) & 1)) ended(1, true);
        was = halves;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h >= halves) break;
          wait(L::kQFull + h, filled[h]++ & 1);
          qk(h, h == halves - 1, n == 1);
        }
        for (int i = 0; i < n && !dead; ++i, ++tl) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h >= halves) break;
            pv(h, tl, i == 0, h == halves - 1);
            if (i + 1 < n) qk(h, h == halves - 1, i + 2 == n);
          }
        }
        if (dead) break;
        ++seg;
      }
      // every issued operation completes before tensor memory is released
      mma_commit(&bars[L::kDrain]);
      mbar_wait_drain(&bars[L::kDrain], 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------------------------------------------------------- scheduler
    // For each segment: the record, and the largest V scale of its blocks.
    int seg = 0;
    bool dead = false;
    const PagedMerge mine = walk_segments(p, range, [&](const Segment& s, const PagedRequest&) {
      uint32_t most = 0u;
      const int32_t* row = a.block_table + (int64_t)s.r * a.MB;
      const int page0 = max(2 * s.kt, s.lo / kBlock), page1 = min(2 * (s.kt + s.n), (s.hi + kBlock - 1) / kBlock);
#pragma unroll 4
      for (int j = page0 + lane; j < page1; j += 32) {
        const int b = __ldg(row + j);
        if (b >= 0 && b < a.NB) most = max(most, __float_as_uint(fabsf(__ldg(a.v_scale + (int64_t)b * a.HK + s.g))));
      }
      most = __reduce_max_sync(kAll, most);
      const int sb = seg % L::kSegs;
      if (seg >= L::kSegs) dead = __any_sync(kAll, !PA_WAIT(L::kSegFree + sb, (seg / L::kSegs + 1) & 1));
      if (dead) return false;
      if (lane == 0) {
        *reinterpret_cast<Segment*>(smem + L::kOffSeg + sb * sizeof(Segment)) = s;
        reinterpret_cast<float*>(smem + L::kOffRef)[sb] = most == 0u ? 1.f : __uint_as_float(most);
        mbar_arrive(&bars[L::kSegFull + sb]);
      }
      __syncwarp();
      ++seg;
      return true;
    });
    if (lane == 0) p.merge[blockIdx.x] = mine;
    const int sb = seg % L::kSegs;
    if (!dead && seg >= L::kSegs) dead = __any_sync(kAll, !PA_WAIT(L::kSegFree + sb, (seg / L::kSegs + 1) & 1));
    if (lane == 0 && !dead) {
      reinterpret_cast<Segment*>(smem + L::kOffSeg + sb * sizeof(Segment))->n = 0;
      mbar_arrive(&bars[L::kSegFull + sb]);
    }
  } else if (warp >= L::kConvWarp0 && warp < L::kSoftWarp0) {
    // ---------------------------------------------------------------- V to f16, times v_scale / R; unseen keys zero
    const int w = warp - L::kConvWarp0;
    // A warp converts its 32 keys in steps of kKeysPer.  8 lanes (what one shared-memory access
    // serves at a time) take 4 chunks of two keys whose numbers differ in bits 0 and 2, so that under the
    // swizzles neither the reads nor the writes meet in a bank.
    constexpr int kHalves = D / 64, kKeysPer = 8 / kHalves;  // 64-column halves of a key; keys a step
    const int ch = (lane & 3) + (D == 128 ? 4 * ((lane >> 3) & 1) : 0);
    const int pair = lane >> (D == 128 ? 4 : 3);              // which two keys of the step's
    Ring<L::kVStages> ring;
    int tl = 0, seg = 0;
    bool dead = false;
    while (true) {
      const int sb = seg % L::kSegs;
      dead = !__all_sync(kAll, PA_WAIT(L::kSegFull + sb, (seg / L::kSegs) & 1));
      if (dead) break;
      const Segment* sp = reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment));
      const int kt = sp->kt, n = sp->n, lo = sp->lo, hi = sp->hi;
      if (n == 0) break;
      const float v_ref = reinterpret_cast<const float*>(smem + L::kOffRef)[sb];
      for (int i = 0; i < n; ++i, ++tl, ring.next()) {
        const int sv = ring.i, vb = tl & 1;
        const bool ok = PA_WAIT(L::kV16Empty + vb, ((tl >> 1) + 1) & 1) &&
                        PA_WAIT(L::kMetaFull + tl % L::kMeta, (tl / L::kMeta) & 1) &&
                        PA_WAIT(L::kVFull + sv, ring.phase);
        dead = !__all_sync(kAll, ok);
        if (dead) break;
        const float* meta = reinterpret_cast<const float*>(smem + L::kOffMeta + (tl % L::kMeta) * 32);
        const float vs = __fdividef(meta[2 + (w >> 1)], v_ref);  // warp w: keys 32 w .. 32 w + 31 of the tile
        const uint32_t f = pack_f16x2(vs, vs);
        const int j0 = (kt + n - 1 - i) * kKeyTile;
        const bool inside = j0 >= lo && j0 + kKeyTile <= hi;  // some row sees each key
        const uint32_t src = smem_u32(smem + L::kOffV + sv * L::kKTile), dst = smem_u32(smem + L::kOffV16 + vb * L::kV16);
#pragma unroll
        for (int it = 0; it < 32 / kKeysPer; ++it) {
          const int first = (it * kKeysPer % 8) / 2 + pair;  // of 8 keys, pairs (0, 5), (1, 4), (2, 7), (3, 6)
          const int r = 32 * w + it * kKeysPer / 8 * 8 + ((lane & 4) ? first ^ 5 : first), j = j0 + r;
          uint32_t c[4], o[8];
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
                       : "r"(src + swz<D>(r, ch))
                       : "memory");
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t x;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(x) : "h"((uint16_t)(c[k >> 1] >> (16 * (k & 1)))));
            o[k] = mul_f16x2(x, f);
          }
          if (!inside && (j < lo || j >= hi)) {
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = 0u;
          }
          // columns 16 ch .. 16 ch + 15 of the key: chunks 2 (ch % 4), + 1 of panel ch / 4, 128-byte swizzle
          const uint32_t base = dst + (uint32_t)(ch >> 2) * (kKeyTile * 128) + r * 128;
          st_shared_v4(base + (((2 * (ch & 3)) ^ (r & 7)) << 4), o[0], o[1], o[2], o[3]);
          st_shared_v4(base + (((2 * (ch & 3) + 1) ^ (r & 7)) << 4), o[4], o[5], o[6], o[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars[L::kV16Full + vb]);
          mbar_arrive(&bars[L::kVEmpty + sv]);
        }
      }
      if (dead) break;
      if (lane == 0) mbar_arrive(&bars[L::kSegFree + sb]);
      ++seg;
    }
  } else if (warp >= L::kSoftWarp0) {
    // ---------------------------------------------------------------- softmax: thread = (half, row, block of the tile)
    const int half = (warp - L::kSoftWarp0) >> 3, blk = ((warp - L::kSoftWarp0) >> 2) & 1, quarter = warp & 3;
    const int row = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t s_addr = tmem + lanes + L::kTmemS + 128 * half + 64 * blk;
    constexpr int kOCols = D / 2;  // columns of O that a thread handles
    const uint32_t o_addr = tmem + lanes + L::kTmemO + 128 * half + kOCols * blk;
    float* red = reinterpret_cast<float*>(smem + L::kOffRed) + half * 2 * kRows;
    float* sums = reinterpret_cast<float*>(smem + L::kOffSum) + half * 2 * kRows;
    const int bar = 1 + 4 * half + quarter;  // the 64 threads of 32 rows
    const float cap = a.softcap * kLog2e;
    int tl = 0, seg = 0, done = 0;  // tiles before the segment; tiles of this half
    bool dead = false;
    // After a wait that ran out the loops go on without waiting to the end of the segment, where the
    // threads of a barrier leave together: none is left behind at one.
    auto wait = [&](int idx, uint32_t parity) {
      const bool ok = !dead && PA_WAIT(idx, parity);
      dead = !__all_sync(kAll, ok);
    };
    while (true) {
      const int sb = seg % L::kSegs;
      wait(L::kSegFull + sb, (seg / L::kSegs) & 1);
      dead = bar_any(bar, 64, dead);
      if (dead) break;
      const Segment* sp = reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment));
      const int kt = sp->kt, n = sp->n;
      if (n == 0) break;
      const float v_ref = reinterpret_cast<const float*>(smem + L::kOffRef)[sb];
      const int heads = sp->heads, ntok = min(sp->ntok - half * half_tokens, half_tokens);  // of this half
      if (ntok <= 0) {  // an empty half
        if (lane == 0) mbar_arrive(&bars[L::kSegFree + sb]);
        tl += n;
        ++seg;
        continue;
      }
      int pos = 0, lo = 0, hi = 0;
      float slope = 0.f, f_row = 0.f;
      int64_t out_row = -1;
      if (row < ntok * heads) {
        PagedRequest q;
        q.load(a, sp->r);
        const int t = sp->t0 + half * half_tokens + row / heads, h = sp->h0 + row % heads;
        pos = q.pos(t);
        lo = q.lo(a, t);
        hi = q.hi(t);
        if (a.alibi_slopes) slope = __ldg(a.alibi_slopes + h) * kLog2e;
        out_row = (int64_t)t * a.H + h;
        f_row = p.q_scale[out_row];
      }
      float m = 0.f, l = 0.f;
      for (int i = 0; i < n; ++i, ++tl, ++done) {
        {
          // S first: a half that skipped segments may be phases of the meta ring behind until then
          const bool ok = !dead && PA_WAIT(L::kSFull + half, done & 1) &&
                          PA_WAIT(L::kMetaFull + tl % L::kMeta, (tl / L::kMeta) & 1);
          dead = !__all_sync(kAll, ok);
        }
        tc_fence_after();
        const float* meta = reinterpret_cast<const float*>(smem + L::kOffMeta + (tl % L::kMeta) * 32);
        const int pages = reinterpret_cast<const int*>(meta)[4];
        const int j0 = (kt + n - 1 - i) * kKeyTile, jb = j0 + 64 * blk;  // first keys of the tile and of this block
        const bool inside = j0 >= sp->all_lo && j0 + kKeyTile <= sp->all_hi && pages == 3;  // no mask
        // the block's keys that this row sees, a bit each
        uint64_t seen = 0ull;
        if (!inside && ((pages >> blk) & 1)) {
          const int lo_k = min(max(lo - jb, 0), 64), hi_k = min(max(hi - jb, 0), 64);
          if (hi_k > lo_k) seen = (~0ull >> (64 - (hi_k - lo_k))) << lo_k;
        }
        float f = f_row * meta[blk];  // (with a cap: over the cap)
        // Where S takes more than a factor, its logits take its place first (in a loop of their own: unrolled into
        // the pass below, the code ran out of the instruction caches).
        if (kBent || !inside) {
          const uint64_t f2 = pack2(f, f);
          uint64_t bend[5];  // cap log2(e) tanh(u) / u by powers of u^2
          if (kBent) {
#pragma unroll
            for (int d = 0; d < 5; ++d) {
              bend[d] = pack2(cap * kTanh[d], cap * kTanh[d]);
              asm volatile("" : "+l"(bend[d]));  // in registers: not made anew at each use
            }
          }
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[16];
            tmem_ld16_sync(s_addr + 16 * c, x);
            // x f, with a cap u = x f / cap
            uint64_t squares = 0ull;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint64_t u2 = mul2(pack2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), f2);
              if (kBent) squares = fma2(u2, u2, squares);
              const float2 u = unpack2(u2);
              x[2 * k] = __float_as_uint(u.x);
              x[2 * k + 1] = __float_as_uint(u.y);
            }
            if (kBent && a.softcap > 0.f) {
              const float2 sq = unpack2(squares);
              if (__all_sync(kAll, sq.x <= kTanhTop && sq.y <= kTanhTop)) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const uint64_t u = pack2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
                  const uint64_t u2 = mul2(u, u);
                  uint64_t y = bend[4];
#pragma unroll
                  for (int d = 3; d >= 0; --d) y = fma2(y, u2, bend[d]);
                  const float2 z = unpack2(mul2(u, y));
                  x[2 * k] = __float_as_uint(z.x);
                  x[2 * k + 1] = __float_as_uint(z.y);
                }
              } else {
                // (each by its own size: another row may have reached its cap, or unseen codes be anything)
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(cap * tanh_any(__uint_as_float(x[k])));
              }
            }
            if (kBent && a.alibi_slopes) {
              const float away = (float)(pos - jb - 16 * c);
#pragma unroll
              for (int k = 0; k < 16; ++k)
                x[k] = __float_as_uint(fmaf(-slope, fabsf(away - (float)k), __uint_as_float(x[k])));
            }
            if (!inside) {
              const uint32_t bits = (uint32_t)(seen >> (16 * c));
#pragma unroll
              for (int k = 0; k < 16; ++k) x[k] = (bits >> k) & 1u ? x[k] : 0xff800000u;  // -infinity
            }
            tmem_st16(s_addr + 16 * c, x);
          }
          tmem_st_wait();
          f = 1.f;
        }
        // logits - m' of keys 16 c .. 16 c + 15 of the block
        auto logits = [&](int c, uint32_t (&x)[16]) {
          tmem_ld16_sync(s_addr + 16 * c, x);
          const uint64_t f2 = pack2(f, f), m2 = pack2(-m, -m);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 y = unpack2(fma2(pack2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), f2, m2));
            x[2 * k] = __float_as_uint(y.x);
            x[2 * k + 1] = __float_as_uint(y.y);
          }
        };
        uint32_t pw[32];  // the weights, f16 pairs
        float part;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
          uint64_t sum2 = 0ull;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t x[16];
            logits(c, x);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float p0 = ex2_approx(__uint_as_float(x[2 * k])), p1 = ex2_approx(__uint_as_float(x[2 * k + 1]));
              sum2 = add2(sum2, pack2(p0, p1));
              pw[8 * c + k] = pack_f16x2(p0, p1);
            }
          }
          const float2 s2 = unpack2(sum2);
          part = s2.x + s2.y;
          // The sum tells whether some weight may be too large for f16, or a row's keys so far too small for it
          // (a sum of 0 with keys to see: below what a float holds).
          const float least = i == kThinAt ? kThin16 : l == 0.f ? kLow16 : 0.f;
          const bool low = l + part < least && (inside || seen != 0ull);
          if (pass == 1 || !bar_any(bar, 64, part > kTop16 || low)) break;
          float top = -INFINITY;  // the largest logit - m'
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[16];
            logits(c, x);
#pragma unroll
            for (int k = 0; k < 16; ++k) top = fmaxf(top, __uint_as_float(x[k]));
          }
          red[blk * kRows + row] = top;
          sums[blk * kRows + row] = l;
          named_bar_sync(bar, 64);
          top = fmaxf(red[row], red[kRows + row]);
          const float before = sums[row] + sums[kRows + row];
          float up = 0.f;
          if (top > kRefresh16 && top < INFINITY)
            up = top - kRefresh16;
          else if (before == 0.f)
            up = top > -INFINITY ? top - kRefresh16 : 0.f;  // (O and l are 0 so far)
          else if (i == kThinAt && before < kThin16)
            up = fmaxf(__log2f(before) - kRefresh16, top - 9.f);
          const float g = before == 0.f ? 1.f : ex2_approx(-up);
          l *= g;
          m += up;
          // P V of the tiles before is complete: S of this tile was issued behind it
          if (i > 0 && __any_sync(kAll, g != 1.f)) {
#pragma unroll
            for (int c = 0; c < kOCols / 16; ++c) {
              uint32_t o[16];
              tmem_ld16_sync(o_addr + 16 * c, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * g);
              tmem_st16(o_addr + 16 * c, o);
            }
          }
        }
        l += part;
        // P over the S that this thread has read
        {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = pw[16 * c + k];
            tmem_st16(s_addr + 16 * c, w);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kPFull + half]);
      }
      // the results: O R / l, or the partial O R with m' and l
      named_bar_sync(bar, 64);
      sums[blk * kRows + row] = l;
      named_bar_sync(bar, 64);
      l += sums[(1 - blk) * kRows + row];
      wait(L::kPvDone + half, (done + 1) & 1);
      tc_fence_after();
      const int slot = sp->slot;
      const int64_t part_at = 2 * (int64_t)blockIdx.x + slot;
      const int c_row = half * half_tokens * heads + row;  // row of the unit
      const float g = slot >= 0 ? v_ref : l == 0.f ? 0.f : v_ref / l;
#pragma unroll
      for (int c = 0; c < kOCols / 16; ++c) {
        uint32_t o[16];
        tmem_ld16_sync(o_addr + 16 * c, o);
        if (out_row < 0 || dead) continue;
        if (slot < 0) {
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            w[k] = pack_bf16x2(__uint_as_float(o[2 * k]) * g, __uint_as_float(o[2 * k + 1]) * g);
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + out_row * D + kOCols * blk + 16 * c);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
          float4* dst = reinterpret_cast<float4*>(p.part_o + (part_at * 256 + c_row) * D + kOCols * blk + 16 * c);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dst[k] = make_float4(__uint_as_float(o[4 * k]) * g, __uint_as_float(o[4 * k + 1]) * g,
                                 __uint_as_float(o[4 * k + 2]) * g, __uint_as_float(o[4 * k + 3]) * g);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars[L::kOFree + half]);
        mbar_arrive(&bars[L::kSegFree + sb]);
      }
      if (blk == 0 && out_row >= 0 && !dead) {
        if (slot < 0) {
          a.lse[out_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        } else {
          p.part_ml[part_at * 512 + c_row] = l == 0.f ? kNoMax : m;
          p.part_ml[part_at * 512 + 256 + c_row] = l;
        }
      }
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

// Workspace: what every call has, then the two terms of q, its scales, and the query tiles' document starts.
size_t terms_offset(const PagedSizes& sz) { return align256(sz.bytes); }
size_t scales_offset(const PagedSizes& sz, int T, int H, int D) {
  return terms_offset(sz) + align256((size_t)2 * T * H * D);
}

size_t docs_offset(const PagedSizes& sz, int T, int H, int D) {
  return scales_offset(sz, T, H, D) + align256((size_t)T * H * 4);
}

// A term of q as [2 T, H, D] bytes (both terms), a box the rows of half a query tile.
cudaError_t term_map(CUtensorMap* m, void* terms, int T, int H, int D, int heads, int tokens) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)2 * T};
  const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)H * D};
  const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)heads, (cuuint32_t)tokens}, es[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, terms, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch(const PagedAttnArgs& a, int num_sms, cudaStream_t stream) {
  using L = PreLay<D>;
  constexpr int C = 2 * kRows;
  const PagedSizes sz = paged_sizes(C, D, L::kPerSm, num_sms);
  uint8_t* terms = static_cast<uint8_t*>(a.workspace) + terms_offset(sz);
  PagedParams p = paged_params<C>(a, sz, kUnitCost);
  p.q_scale = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + scales_offset(sz, a.T, a.H, D));
  CUtensorMap k_map, v_map, q_map;
  cudaError_t e = cache_maps(a, &k_map, &v_map);
  if (e == cudaSuccess) e = term_map(&q_map, terms, a.T, a.H, D, p.Gr, p.tq / 2);
  if (e != cudaSuccess) return e;
  const int64_t threads = (int64_t)a.T * a.H * (D / 8);
  e = launch_overlapped(paged_split_q_kernel<D>, dim3((unsigned)((threads + kSplitThreads - 1) / kSplitThreads)),
                        kSplitThreads, 0, stream, a, terms, p.q_scale);
  if (e == cudaSuccess && a.doc_start) {
    int32_t* docs = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(a.workspace) + docs_offset(sz, a.T, a.H, D));
    const int slots = a.T / p.tq + a.R;
    e = launch_overlapped(paged_tile_doc_kernel, dim3((unsigned)((slots + kSplitThreads / 32 - 1) / (kSplitThreads / 32))),
                          kSplitThreads, 0, stream, p, docs, slots);
    p.tile_doc = docs;
  }
  if (e == cudaSuccess)
    e = launch_overlapped(a.softcap > 0.f || a.alibi_slopes ? paged_prefill_kernel<D, true> : paged_prefill_kernel<D, false>,
                          dim3((unsigned)p.ctas), L::kThreads, L::kSmem, stream, p, k_map, v_map, q_map);
  return e == cudaSuccess ? launch_merge<D, C>(p, stream) : e;
}

}  // namespace

size_t paged_prefill_workspace(int T, int H, int D, int R, int num_sms) {
  return docs_offset(paged_sizes(2 * kRows, D, 1, num_sms), T, H, D) + ((size_t)T + R) * 4;
}

cudaError_t launch_paged_prefill(const PagedAttnArgs& a, int num_sms, cudaStream_t stream) {
  return a.D == 128 ? launch<128>(a, num_sms, stream) : launch<64>(a, num_sms, stream);
}

cudaError_t paged_prefill_timed_out(int** word) { return timed_out_word(word); }
cudaError_t paged_prefill_wait_check(int* status, cudaStream_t stream) { return wait_check(status, stream); }

}  // namespace smla
