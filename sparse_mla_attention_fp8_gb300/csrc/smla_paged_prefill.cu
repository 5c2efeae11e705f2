// Attention over the paged 8-bit K/V cache for many rows per K/V head: prompts,
// chunks of them, and many heads per K/V head.  What is computed and how the
// call is cut into segments: smla_paged_attn.cu, smla_paged.cuh.
//
// A query tile has 2 x 128 rows (tokens x heads of one K/V head); each half
// meets every key tile of 128 keys in two products of 128 x 128 x D, so the
// tensor cores bound it, with the softmax and the shared memory that feeds the
// products close behind.  One half's softmax runs under the other's products.
//  * S [row][key] = Q K^T on the codes as stored (kind::f8f6f4), q in two e4m3
//    terms (exact but for components below 2^-10 of their row's largest): two
//    passes at the 8-bit rate cost what one at the 16-bit rate would, without
//    converting K.
//  * O += P V in f16 (kind::f16): P then needs one conversion per pair, where two
//    8-bit terms need five, and V is converted once for the 256 rows.  The
//    conversion also applies v_scale / R (R the largest v_scale of the segment:
//    at most 1) and zeroes the keys that no row sees, whose codes may be
//    anything.  P <= 2^15 keeps 11 bits down to 2^-14 and loses nothing above
//    2^-25.
//  * Softmax: thread pair = row, each thread the keys of one block (one K
//    scale).  P = 2^(x - m') with the row's running reference m', computed in one
//    pass over S into registers; only if some weight passes 2^15 is m' refreshed
//    (to put the tile's largest at 2^2), O scaled in tensor memory and the pass
//    repeated.
//  * P overwrites S in tensor memory and enters P V from there.
//  * Roles: TMA producer, MMA issuer, scheduler, 4 warps converting V, 8 softmax
//    warps per half, which also split Q and write the results.
#include "smla_paged.cuh"

namespace smla {

namespace {

constexpr int kRows = 128;          // rows of a half
constexpr float kTop16 = 15.f;      // P = 2^(x - m') <= 2^15 (f16: 65504)
constexpr float kRefresh16 = 2.f;   // a refreshed m' puts the tile's maximum at 2^2

// (a.x, a.y) * (b.x, b.y) + (c.x, c.y) and sums, two at a time.
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
  static constexpr int kMeta = 2 * kStages;                 // ring of block scales and flags
  static constexpr int kQTerm = kRows * D, kQHalf = 2 * kQTerm;
  static constexpr int kSegs = 2;
  static constexpr int kOffV = kStages * kKTile;
  static constexpr int kOffV16 = kOffV + kVStages * kKTile;
  static constexpr int kOffQ = kOffV16 + 2 * kV16;
  static constexpr int kOffMeta = kOffQ + 2 * kQHalf;
  static constexpr int kOffRed = kOffMeta + kMeta * 32;            // float [2 halves][2][128] maxima
  static constexpr int kOffSum = kOffRed + 4 * kRows * 4;          // float [2 halves][2][128] sums, and Q's maxima
  static constexpr int kOffRef = kOffSum + 4 * kRows * 4;          // float [segs] largest v scale
  static constexpr int kOffSeg = kOffRef + 16;
  static constexpr int kOffBar = (kOffSeg + kSegs * (int)sizeof(Segment) + 7) / 8 * 8;
  enum {
    kKFull = 0, kKEmpty = kKFull + kStages, kVFull = kKEmpty + kStages, kVEmpty = kVFull + kVStages,
    kMetaFull = kVEmpty + kVStages, kV16Full = kMetaFull + kMeta, kV16Empty = kV16Full + 2, kSFull = kV16Empty + 2,
    kPFull = kSFull + 2, kPvDone = kPFull + 2, kQFull = kPvDone + 2, kSegFull = kQFull + 2,
    kSegFree = kSegFull + kSegs, kDrain = kSegFree + kSegs, kNumBars
  };
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmem = kOffMisc + 16 + 1024;
  static constexpr int kTmemS = 0, kTmemO = 256, kTmemCols = 512;  // S of the halves, O of the halves: 128 columns each
  static_assert(kSmem <= 232448, "shared memory");
  static_assert((kMaxPagedRequests + 1 + kWarps) * 8 <= kOffMeta, "prefix sums fit the operands' memory");
  static_assert(kKTile % 1024 == 0 && kV16 % 1024 == 0 && kQTerm % 1024 == 0, "operand alignment");
};

template <int D>
__global__ void __launch_bounds__(PreLay<D>::kThreads, PreLay<D>::kPerSm)
    paged_prefill_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map) {
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
      mbar_init(&bars[L::kQFull + i], 8);
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
        const float k0 = __shfl_sync(kAll, ks, at + 1), k1 = __shfl_sync(kAll, ks, at);
        const float v0 = __shfl_sync(kAll, vs, at + 1), v1 = __shfl_sync(kAll, vs, at);
        const int st = tl % L::kStages, use = tl / L::kStages, sv = tl % L::kVStages, vuse = tl / L::kVStages;
        if (use > 0) dead = __any_sync(kAll, !PA_WAIT(L::kKEmpty + st, (use + 1) & 1));
        if (dead) break;
        const int y0 = b0 >= 0 ? (b0 * a.HK + s.g) * kBlock : outside;
        const int y1 = b1 >= 0 ? (b1 * a.HK + s.g) * kBlock : outside;
        if (lane == 0) {
          // slot tl % kMeta: its tile before had its S read before the K stage was free twice
          float* meta = reinterpret_cast<float*>(smem + L::kOffMeta + (tl % L::kMeta) * 32);
          *reinterpret_cast<float4*>(meta) = make_float4(k0, k1, v0, v1);
          reinterpret_cast<int*>(meta)[4] = (b0 >= 0 ? 1 : 0) | (b1 >= 0 ? 2 : 0);
          mbar_arrive(&bars[L::kMetaFull + tl % L::kMeta]);
          const uint32_t kd = smem_u32(smem + st * L::kKTile);
          mbar_arrive_expect_tx(&bars[L::kKFull + st], L::kKTile);
          tma_load_2d(kd, &k_map, 0, y0, &bars[L::kKFull + st]);
          tma_load_2d(kd + kBlock * D, &k_map, 0, y1, &bars[L::kKFull + st]);
        }
        __syncwarp();
        if (vuse > 0) dead = __any_sync(kAll, !PA_WAIT(L::kVEmpty + sv, (vuse + 1) & 1));
        if (lane == 0 && !dead) {
          const uint32_t vd = smem_u32(smem + L::kOffV + sv * L::kKTile);
          mbar_arrive_expect_tx(&bars[L::kVFull + sv], L::kKTile);
          tma_load_2d(vd, &v_map, 0, y0, &bars[L::kVFull + sv]);
          tma_load_2d(vd + kBlock * D, &v_map, 0, y1, &bars[L::kVFull + sv]);
        }
        __syncwarp();
        if (dead) {  // this tile's K copies are in flight, its V copies are not
          mbar_wait_drain(&bars[L::kKFull + st], use & 1);
          break;
        }
      }
      if (dead) break;
      if (lane == 0) mbar_arrive(&bars[L::kSegFree + sb]);
      ++seg;
    }
    // no copy may still be landing when the CTA exits
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
      bool dead = false;
      auto wait = [&](int idx, uint32_t parity) {
        if (!dead) dead = !PA_WAIT(idx, parity);
        return !dead;
      };
      auto qk = [&](int h, int t, bool last) {
        const int st = t % L::kStages;
        if (!wait(L::kKFull + st, (t / L::kStages) & 1)) return;
        if (done[h] > 0 && !wait(L::kPvDone + h, (done[h] + 1) & 1)) return;
        tc_fence_after();
        const uint64_t dk = dk0 + (uint64_t)((st * L::kKTile) >> 4), dq = dq0 + (uint64_t)((h * L::kQHalf) >> 4);
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            mma_f8(tmem + L::kTmemS + 128 * h, dq + ((term * L::kQTerm + 32 * k) >> 4), dk + ((32 * k) >> 4), id_qk,
                   term + k > 0 ? 1u : 0u);
        mma_commit(&bars[L::kSFull + h]);
        if (last) mma_commit(&bars[L::kKEmpty + st]);
      };
      auto pv = [&](int h, int t, bool first, bool last) {
        const int vb = t & 1;
        if (!wait(L::kPFull + h, done[h] & 1) || !wait(L::kV16Full + vb, (t >> 1) & 1)) return;
        tc_fence_after();
        const uint64_t dv = dv0 + (uint64_t)((vb * L::kV16) >> 4);
#pragma unroll
        for (int k = 0; k < kKeyTile / 16; ++k)  // P: block b's 64 keys in columns 64 b .. 64 b + 31
          mma_ts(tmem + L::kTmemO + 128 * h, tmem + L::kTmemS + 128 * h + 64 * (k >> 2) + 8 * (k & 3),
                 dv + ((2048 * k) >> 4), id_pv, (!first || k > 0) ? 1u : 0u);
        mma_commit(&bars[L::kPvDone + h]);
        if (last) mma_commit(&bars[L::kV16Empty + vb]);
        ++done[h];
      };
      while (true) {
        const int sb = seg % L::kSegs;
        if (!wait(L::kSegFull + sb, (seg / L::kSegs) & 1)) break;
        const Segment* sp = reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment));
        const int n = sp->n, halves = sp->ntok > half_tokens ? 2 : 1;
        if (n == 0) break;
        mbar_arrive(&bars[L::kSegFree + sb]);
        // the halves' Q is split, and their O of the segment before has been read
        for (int h = 0; h < halves; ++h) wait(L::kQFull + h, filled[h]++ & 1);
        for (int h = 0; h < halves; ++h) qk(h, tl, h == halves - 1);
        for (int i = 0; i < n && !dead; ++i, ++tl)
          for (int h = 0; h < halves; ++h) {
            pv(h, tl, i == 0, h == halves - 1);
            if (i + 1 < n) qk(h, tl + 1, h == halves - 1);
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
    const PagedMerge mine = walk_segments(p, range, [&](const Segment& s) {
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
    constexpr int kChunks = D / 16;            // 16-byte chunks of a key's codes
    constexpr int kKeysPer = 32 / kChunks;     // keys that a warp converts at a time
    const int ch = lane % kChunks, sub = lane / kChunks;
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
      for (int i = 0; i < n; ++i, ++tl) {
        const int sv = tl % L::kVStages, vb = tl & 1;
        const bool ok = (tl < 2 || PA_WAIT(L::kV16Empty + vb, ((tl >> 1) + 1) & 1)) &&
                        PA_WAIT(L::kMetaFull + tl % L::kMeta, (tl / L::kMeta) & 1) &&
                        PA_WAIT(L::kVFull + sv, (tl / L::kVStages) & 1);
        dead = !__all_sync(kAll, ok);
        if (dead) break;
        const float* meta = reinterpret_cast<const float*>(smem + L::kOffMeta + (tl % L::kMeta) * 32);
        const float vs = __fdividef(meta[2 + (w >> 1)], v_ref);  // warp w: keys 32 w .. 32 w + 31 of the tile
        const uint32_t f = pack_f16x2(vs, vs);
        const int j0 = (kt + n - 1 - i) * kKeyTile;
        const uint32_t src = smem_u32(smem + L::kOffV + sv * L::kKTile), dst = smem_u32(smem + L::kOffV16 + vb * L::kV16);
#pragma unroll
        for (int it = 0; it < 32 / kKeysPer; ++it) {
          const int r = 32 * w + it * kKeysPer + sub, j = j0 + r;
          uint32_t c[4], o[8];
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
                       : "r"(src + swz<D>(r, ch))
                       : "memory");
          const bool seen = j >= lo && j < hi;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t x;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(x) : "h"((uint16_t)(c[k >> 1] >> (16 * (k & 1)))));
            o[k] = seen ? mul_f16x2(x, f) : 0u;
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
    const float cap_to = a.softcap > 0.f ? 2.f * kLog2e / a.softcap : 0.f, cap = a.softcap * kLog2e;
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
      float slope = 0.f, f_row;
      int64_t out_row = -1;
      {
        // this row, and this thread's half of its Q in two terms
        const uint4* src = nullptr;
        if (row < ntok * heads) {
          PagedRequest q;
          q.load(a, sp->r);
          const int t = sp->t0 + half * half_tokens + row / heads, h = sp->h0 + row % heads;
          pos = q.pos(t);
          lo = q.lo(a, t);
          hi = q.hi(t);
          if (a.alibi_slopes) slope = __ldg(a.alibi_slopes + h) * kLog2e;
          out_row = (int64_t)t * a.H + h;
          src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (int64_t)t * a.q_stride +
                                               (int64_t)h * D + blk * (D / 2));
        }
        uint4 v[D / 16];
        uint32_t amax = 0u;  // of the magnitudes' bits
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          v[i] = src ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) amax = max(amax, max((w[k] << 16) & 0x7fffffffu, w[k] & 0x7fff0000u));
        }
        reinterpret_cast<uint32_t*>(red)[blk * kRows + row] = amax;
        named_bar_sync(bar, 64);
        amax = max(amax, reinterpret_cast<const uint32_t*>(red)[(1 - blk) * kRows + row]);
        named_bar_sync(bar, 64);
        // 2^sh: amax = (1 + f) 2^e to at most 448 = 1.75 * 2^8
        int sh = 8 - ((int)(amax >> 23) - 127) - ((amax & 0x7fffffu) > 0x600000u);
        sh = amax == 0u ? 0 : min(sh, 120);
        const float f = __uint_as_float((uint32_t)(sh + 127) << 23);
        // a row with an infinity or NaN has no finite result
        f_row = amax >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 - sh) << 23);
        f_row *= a.sm_scale * (a.softcap > 0.f ? 1.f : kLog2e);
        const uint32_t qd = smem_u32(smem + L::kOffQ + half * L::kQHalf);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {  // 16 codes each
          const uint32_t w[8] = {v[2 * i].x,     v[2 * i].y,     v[2 * i].z,     v[2 * i].w,
                                 v[2 * i + 1].x, v[2 * i + 1].y, v[2 * i + 1].z, v[2 * i + 1].w};
          uint32_t hc[4] = {0u, 0u, 0u, 0u}, lc[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float y0 = __uint_as_float(w[k] << 16) * f, y1 = __uint_as_float(w[k] & 0xffff0000u) * f;
            const uint32_t c = e4m3x2(y0, y1);
            const float2 back = e4m3x2_f32(c);
            hc[k >> 1] |= c << (16 * (k & 1));
            lc[k >> 1] |= e4m3x2(y0 - back.x, y1 - back.y) << (16 * (k & 1));
          }
          const uint32_t dst = qd + swz<D>(row, blk * (D / 32) + i);
          st_shared_v4(dst, hc[0], hc[1], hc[2], hc[3]);
          st_shared_v4(dst + L::kQTerm, lc[0], lc[1], lc[2], lc[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();  // O of the segment before has been read
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kQFull + half]);
      }
      float m = kNoMax, l = 0.f;
      for (int i = 0; i < n; ++i, ++tl, ++done) {
        {
          // S first: a half that skipped segments may be phases of the meta ring behind until then
          const bool ok = !dead && PA_WAIT(L::kSFull + half, done & 1) &&
                          PA_WAIT(L::kMetaFull + tl % L::kMeta, (tl / L::kMeta) & 1);
          dead = !__all_sync(kAll, ok);
        }
        tc_fence_after();
        const float* meta = reinterpret_cast<const float*>(smem + L::kOffMeta + (tl % L::kMeta) * 32);
        const float f = f_row * meta[blk];
        const int pages = reinterpret_cast<const int*>(meta)[4];
        const int j0 = (kt + n - 1 - i) * kKeyTile, jb = j0 + 64 * blk;  // first keys of the tile and of this block
        const bool inside = j0 >= sp->all_lo && j0 + kKeyTile <= sp->all_hi && pages == 3;  // no mask
        const bool plain = inside && !a.alibi_slopes && !(a.softcap > 0.f);
        // visible keys of the block for this row: lo_k <= k < lo_k + n_k
        const int lo_k = max(lo - jb, 0), n_k = (pages >> blk) & 1 ? max(min(hi - jb, 64) - lo_k, 0) : 0;
        uint32_t pw[32];  // the weights, f16 pairs
        float part;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
          const float base = m == kNoMax ? 0.f : m;
          float top = -INFINITY;  // the largest x - base
          uint64_t sum2 = 0ull;
          // weights of the 16 keys x - base; two sums and the largest besides
          auto weigh = [&](const uint32_t (&x)[16], int c) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float x0 = __uint_as_float(x[2 * k]), x1 = __uint_as_float(x[2 * k + 1]);
              top = fmaxf(top, fmaxf(x0, x1));
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              sum2 = add2(sum2, pack2(p0, p1));
              pw[8 * c + k] = pack_f16x2(p0, p1);
            }
          };
          if (plain) {
            const uint64_t f2 = pack2(f, f), m2 = pack2(-base, -base);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t x[16];
              tmem_ld16_sync(s_addr + 16 * c, x);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float2 y = unpack2(fma2(pack2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), f2, m2));
                x[2 * k] = __float_as_uint(y.x);
                x[2 * k + 1] = __float_as_uint(y.y);
              }
              weigh(x, c);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t x[16];
              tmem_ld16_sync(s_addr + 16 * c, x);
#pragma unroll
              for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * f);
              if (a.softcap > 0.f) {
                // cap tanh(x / cap) = cap (1 - 2 / (1 + e^(2 x / cap))), to within a few 2^-23 cap
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  x[k] = __float_as_uint(
                      fmaf(-2.f * cap, __fdividef(1.f, 1.f + ex2_approx(__uint_as_float(x[k]) * cap_to)), cap));
              }
              if (a.alibi_slopes) {
                float away = (float)(pos - jb - 16 * c);
                asm volatile("" : "+f"(away));  // as lo_c below
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  x[k] = __float_as_uint(fmaf(-slope, fabsf(away - (float)k), __uint_as_float(x[k])));
              }
              if (!inside) {
                // (opaque: otherwise the 64 comparisons move out of the pass loop and run for every tile)
                int lo_c = 16 * c - lo_k;
                asm volatile("" : "+r"(lo_c));
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  x[k] = (uint32_t)(lo_c + k) < (uint32_t)n_k ? x[k] : 0xff800000u;  // -infinity
              }
#pragma unroll
              for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) - base);
              weigh(x, c);
            }
          }
          const float2 s2 = unpack2(sum2);
          part = s2.x + s2.y;
          if (pass == 1 || !bar_any(bar, 64, top + (base - m) > kTop16)) break;
          // a weight too large for f16, or a row's first key: refresh the row's reference
          red[blk * kRows + row] = top == top ? top + base : -INFINITY;
          named_bar_sync(bar, 64);
          top = fmaxf(red[row], red[kRows + row]);
          float g = 1.f;
          if (top - m > kTop16) {
            const float to = top - kRefresh16;
            g = ex2_approx(m - to);
            l *= g;
            m = to;
          }
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
      if (blk == 0 && out_row >= 0 && !dead) {
        if (slot < 0) {
          a.lse[out_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        } else {
          p.part_ml[part_at * 512 + c_row] = m;
          p.part_ml[part_at * 512 + 256 + c_row] = l;
        }
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

template <int D>
cudaError_t launch(const PagedAttnArgs& a, int num_sms, cudaStream_t stream) {
  using L = PreLay<D>;
  return launch_paged<D, 2 * kRows>(paged_prefill_kernel<D>, a, L::kPerSm, L::kThreads, L::kSmem, num_sms, stream);
}

}  // namespace

cudaError_t launch_paged_prefill(const PagedAttnArgs& a, int num_sms, cudaStream_t stream) {
  return a.D == 128 ? launch<128>(a, num_sms, stream) : launch<64>(a, num_sms, stream);
}

}  // namespace smla
