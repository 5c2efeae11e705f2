// Attention over the paged 8-bit K/V cache for many rows per K/V head: prompts,
// chunks of them, and many heads per K/V head.  What is computed and how the
// call is cut into segments: smla_paged_attn.cu, smla_paged.cuh.
//
// A query tile has 128 rows (tokens x heads of one K/V head), which meet each
// key tile of 128 keys in two products of 128 x 128 x D: the tensor cores bound
// it, with the softmax close behind, so two CTAs share an SM and one's softmax
// runs under the other's products.
//  * The codes enter both products as stored (kind::f8f6f4), twice each: q in
//    two e4m3 terms (exact but for components below 2^-10 of their row's
//    largest), P in an e4m3 and an e5m2 term (remainder) into the same sums:
//    7 to 8 significant bits down to P = 2^-6, nothing lost above 2^-16.  Two
//    passes at the 8-bit rate cost what one at the 16-bit rate would, without
//    converting K or V.
//  * S [row][key] = Q K^T: thread pair = row, each thread the keys of one block
//    (one K scale).  S is read twice, first for the maximum (the tile's largest
//    logit is checked against the row's reference m', as in smla_paged_attn.cu),
//    then in halves for the weights: 32 values at a time stay in registers.
//  * P overwrites the S columns that its thread has read and enters P V from
//    tensor memory.  V scales: P carries v_scale / R, R the largest of the
//    segment, so O accumulates in tensor memory over the segment; it is scaled
//    there in the rare tiles that refresh a row's m'.
//  * Roles: TMA producer, MMA issuer, scheduler, 8 softmax warps, which also
//    split Q and write the results.
#include "smla_paged.cuh"

namespace smla {

namespace {

constexpr int kRows = 128;

// A [M, K] from tensor memory, B [N, K] from shared memory.
__device__ __forceinline__ void mma_f8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}" ::"r"(
          d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Two weights -> e4m3 codes and e5m2 codes of the remainders (low byte from
// x0), split in f16x2: 11 bits, more than the two terms keep.
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

template <int D>
struct PreLay {
  static constexpr int kWarps = 12, kThreads = 32 * kWarps, kPerSm = 2;
  static constexpr int kKTile = kKeyTile * D;
  static constexpr int kStage = 2 * kKTile;
  static constexpr int kStages = 2 * (128 / D);
  static constexpr int kMeta = kStages + 2;
  static constexpr int kQTerm = kRows * D;
  static constexpr int kSegs = 2;
  static constexpr int kOffQ = kStages * kStage;
  static constexpr int kOffMeta = kOffQ + 2 * kQTerm;
  static constexpr int kOffRed = kOffMeta + kMeta * 32;            // float [2][128] maxima
  static constexpr int kOffSum = kOffRed + 2 * kRows * 4;          // float [2][128] sums, and Q's maxima
  static constexpr int kOffRef = kOffSum + 2 * kRows * 4;          // float [segs] largest v scale
  static constexpr int kOffSeg = kOffRef + 16;
  static constexpr int kOffBar = (kOffSeg + kSegs * (int)sizeof(Segment) + 7) / 8 * 8;
  enum {
    kKFull = 0, kVFull = kKFull + kStages, kEmpty = kVFull + kStages, kSFull = kEmpty + kStages, kPFull, kPvDone, kQFull,
    kSegFull, kSegFree = kSegFull + kSegs, kDrain = kSegFree + kSegs, kNumBars
  };
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmem = kOffMisc + 16 + 1024;
  static constexpr int kTmemS = 0, kTmemO = 128, kTmemCols = 256;
  static_assert(kPerSm * (kSmem + 1024) <= 233472 && kPerSm * kTmemCols <= 512, "two CTAs per SM");
  static_assert((kMaxPagedRequests + 1 + kWarps) * 8 <= kOffMeta, "prefix sums fit the stages and Q");
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

  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&bars[L::kKFull + i], 1);
      mbar_init(&bars[L::kVFull + i], 1);
      mbar_init(&bars[L::kEmpty + i], 1);
    }
    mbar_init(&bars[L::kSFull], 1);
    mbar_init(&bars[L::kPFull], 8);
    mbar_init(&bars[L::kPvDone], 1);
    mbar_init(&bars[L::kQFull], 8);
    for (int i = 0; i < L::kSegs; ++i) {
      mbar_init(&bars[L::kSegFull + i], 1);
      mbar_init(&bars[L::kSegFree + i], 2 + 8);
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
        const float k0 = __shfl_sync(kAll, ks, at + 1), k1 = __shfl_sync(kAll, ks, at);
        const float v0 = __shfl_sync(kAll, vs, at + 1), v1 = __shfl_sync(kAll, vs, at);
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
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t id_qk = idesc_e4m3(128, kKeyTile, 0, 0);
      constexpr uint32_t id_hi = idesc_e4m3(128, D, 0, 1);
      constexpr uint32_t id_lo = id_hi | (1u << 7);  // A = e5m2
      constexpr uint32_t lay = D == 128 ? kLayoutSw128 : kLayoutSw64;
      const uint64_t dk0 = make_sdesc(smem_u32(smem), 16, 8 * D, lay);
      const uint64_t dv0 = make_sdesc(smem_u32(smem + L::kKTile), 0, 8 * D, lay);  // read MN-major: one D-byte atom
      const uint64_t dq = make_sdesc(smem_u32(smem + L::kOffQ), 16, 8 * D, lay);
      int tl = 0, seg = 0;
      bool dead = false;
      while (!dead) {
        const int sb = seg % L::kSegs;
        if (!PA_WAIT(L::kSegFull + sb, (seg / L::kSegs) & 1)) break;
        const int n = reinterpret_cast<const Segment*>(smem + L::kOffSeg + sb * sizeof(Segment))->n;
        if (n == 0) break;
        mbar_arrive(&bars[L::kSegFree + sb]);
        if (!PA_WAIT(L::kQFull, seg & 1)) break;  // and the previous segment's O has been read
        for (int i = 0; i < n; ++i, ++tl) {
          const int st = tl % L::kStages;
          // S overwrites the P that the previous tile's product reads
          if (!PA_WAIT(L::kKFull + st, (tl / L::kStages) & 1) || (tl > 0 && !PA_WAIT(L::kPvDone, (tl + 1) & 1))) {
            dead = true;
            break;
          }
          tc_fence_after();
          const uint64_t dk = dk0 + (uint64_t)((st * L::kStage) >> 4), dv = dv0 + (uint64_t)((st * L::kStage) >> 4);
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              mma_f8(tmem + L::kTmemS, dq + ((term * L::kQTerm + 32 * k) >> 4), dk + ((32 * k) >> 4), id_qk,
                     term + k > 0 ? 1u : 0u);
          mma_commit(&bars[L::kSFull]);
          if (!PA_WAIT(L::kPFull, tl & 1) || !PA_WAIT(L::kVFull + st, (tl / L::kStages) & 1)) {
            dead = true;
            break;
          }
          tc_fence_after();
          // P: block b's 64 keys in columns 64 b: 16 of first terms, 16 of second ones (4 keys a column)
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f8_ts(tmem + L::kTmemO, tmem + L::kTmemS + 64 * (k >> 1) + 16 * term + 8 * (k & 1),
                        dv + ((32 * D * k) >> 4), term ? id_lo : id_hi, (i > 0 || term + k > 0) ? 1u : 0u);
          mma_commit(&bars[L::kEmpty + st]);
          mma_commit(&bars[L::kPvDone]);
        }
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
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax: thread = (row, block of the tile)
    const int blk = (warp - 4) >> 2, quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t s_addr = tmem + lanes + L::kTmemS + 64 * blk;
    constexpr int kOCols = D / 2;  // columns of O that a thread handles
    const uint32_t o_addr = tmem + lanes + L::kTmemO + kOCols * blk;
    float* red = reinterpret_cast<float*>(smem + L::kOffRed);
    float* sums = reinterpret_cast<float*>(smem + L::kOffSum);
    const int bar = 1 + quarter;  // the 64 threads of 32 rows
    const float cap_to = a.softcap > 0.f ? 2.f * kLog2e / a.softcap : 0.f, cap = a.softcap * kLog2e;
    auto capped = [&](float x) {  // cap tanh(x / cap), to within a few 2^-23 cap
      return fmaf(-2.f * cap, __fdividef(1.f, 1.f + ex2_approx(x * cap_to)), cap);
    };
    int tl = 0, seg = 0;
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
      int pos = 0, lo = 0, hi = 0;
      float slope = 0.f, f_row;
      int64_t out_row = -1;
      {
        // this row, and this thread's half of its Q in two terms
        const int heads = sp->heads;
        const uint4* src = nullptr;
        if (row < sp->ntok * heads) {
          PagedRequest q;
          q.load(a, sp->r);
          const int t = sp->t0 + row / heads, h = sp->h0 + row % heads;
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
        named_bar_sync(bar, 64);  // the last segment's sums have been read
        reinterpret_cast<uint32_t*>(sums)[blk * kRows + row] = amax;
        named_bar_sync(bar, 64);
        amax = max(amax, reinterpret_cast<const uint32_t*>(sums)[(1 - blk) * kRows + row]);
        // 2^sh: amax = (1 + f) 2^e to at most 448 = 1.75 * 2^8
        int sh = 8 - ((int)(amax >> 23) - 127) - ((amax & 0x7fffffu) > 0x600000u);
        sh = amax == 0u ? 0 : min(sh, 120);
        const float f = __uint_as_float((uint32_t)(sh + 127) << 23);
        // a row with an infinity or NaN has no finite result
        f_row = amax >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 - sh) << 23);
        f_row *= a.sm_scale * (a.softcap > 0.f ? 1.f : kLog2e);
        const uint32_t qd = smem_u32(smem + L::kOffQ);
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
        if (lane == 0) mbar_arrive(&bars[L::kQFull]);
      }
      float m = kNoMax, l = 0.f;
      for (int i = 0; i < n; ++i, ++tl) {
        const int st = tl % L::kStages;
        {
          // the tile's scales and flags (behind its K copies), and its S
          const bool ok = !dead && PA_WAIT(L::kKFull + st, (tl / L::kStages) & 1) && PA_WAIT(L::kSFull, tl & 1);
          dead = !__all_sync(kAll, ok);
        }
        tc_fence_after();
        const float* meta = reinterpret_cast<const float*>(smem + L::kOffMeta + (tl % L::kMeta) * 32);
        const float f = f_row * meta[blk], vf = __fdividef(meta[2 + blk], v_ref);
        const int pages = reinterpret_cast<const int*>(meta)[4];
        const int j0 = (kt + n - 1 - i) * kKeyTile, jb = j0 + 64 * blk;  // first keys of the tile and of this block
        const bool inside = j0 >= sp->all_lo && j0 + kKeyTile <= sp->all_hi && pages == 3;  // no mask
        const bool plain = inside && !a.alibi_slopes;
        const int lo_k = (pages >> blk) & 1 ? lo - jb : 64, hi_k = hi - jb;  // visible: lo_k <= k < hi_k
        // the logits of keys 32 c .. 32 c + 31 of the block
        auto logits = [&](int c, float (&x)[32]) {
          uint32_t raw[32];
          tmem_ld32_sync(s_addr + 32 * c, raw);
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(raw[k]) * f;
          if (a.softcap > 0.f) {
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = capped(x[k]);
          }
          if (a.alibi_slopes) {
            const float away = (float)(pos - jb - 32 * c);
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = fmaf(-slope, fabsf(away - (float)k), x[k]);
          }
          if (!inside) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (32 * c + k < lo_k || 32 * c + k >= hi_k) x[k] = -INFINITY;
          }
        };
        float top = -INFINITY;
        if (plain) {
          // the largest logit comes from the largest product (the smallest under a negative scale)
          float most = -INFINITY, least = INFINITY;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t raw[32];
            tmem_ld32_sync(s_addr + 32 * c, raw);
            if (f >= 0.f) {
#pragma unroll
              for (int k = 0; k < 32; ++k) most = fmaxf(most, __uint_as_float(raw[k]));
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k) least = fminf(least, __uint_as_float(raw[k]));
            }
          }
          top = f >= 0.f ? most * f : least * f;
          if (a.softcap > 0.f) top = capped(top);
        } else {
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            float x[32];
            logits(c, x);
#pragma unroll
            for (int k = 0; k < 32; ++k) top = fmaxf(top, x[k]);
          }
        }
        if (bar_any(bar, 64, top - m > kTop)) {
          red[blk * kRows + row] = top == top ? top : -INFINITY;
          named_bar_sync(bar, 64);
          top = fmaxf(red[row], red[kRows + row]);
          float g = 1.f;
          if (top - m > kTop) {
            const float to = top - kRefresh;
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
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          float x[32];
          if (plain && !(a.softcap > 0.f)) {
            uint32_t raw[32];
            tmem_ld32_sync(s_addr + 32 * c, raw);
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = fmaf(__uint_as_float(raw[k]), f, -m);
          } else {
            logits(c, x);
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] -= m;
          }
          uint32_t hw[8], lw[8];
          float part = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t h0, l0, h1, l1;
            const float p0 = ex2_approx(x[4 * k]), p1 = ex2_approx(x[4 * k + 1]);
            const float p2 = ex2_approx(x[4 * k + 2]), p3 = ex2_approx(x[4 * k + 3]);
            part += (p0 + p1) + (p2 + p3);
            split_p(p0 * vf, p1 * vf, h0, l0);
            split_p(p2 * vf, p3 * vf, h1, l1);
            hw[k] = h0 | (h1 << 16);
            lw[k] = l0 | (l1 << 16);
          }
          l += part;
          tmem_st8(s_addr + 8 * c, hw);
          tmem_st8(s_addr + 16 + 8 * c, lw);
        }
        if (!inside) {
          // keys that no row sees may hold any codes: their V rows become zeros (two threads a row)
          const int key = (32 * (4 * blk + quarter) + lane) >> 1, j = j0 + key;
          const bool zero_v = j < sp->lo || j >= sp->hi;
          if (__any_sync(kAll, zero_v)) {
            wait(L::kVFull + st, (tl / L::kStages) & 1);
            if (zero_v) {
              const uint32_t vd = smem_u32(smem + st * L::kStage + L::kKTile) + key * D + (lane & 1) * (D / 2);
#pragma unroll
              for (int k = 0; k < D / 32; ++k) st_shared_v4(vd + 16 * k, 0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::kPFull]);
      }
      // the results: O R / l, or the partial O R with m' and l
      named_bar_sync(bar, 64);  // Q's maxima have been read
      sums[blk * kRows + row] = l;
      named_bar_sync(bar, 64);
      l += sums[(1 - blk) * kRows + row];
      wait(L::kPvDone, (tl + 1) & 1);
      tc_fence_after();
      const int slot = sp->slot;
      const int64_t part = 2 * (int64_t)blockIdx.x + slot;
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
          float4* dst = reinterpret_cast<float4*>(p.part_o + (part * kRows + row) * D + kOCols * blk + 16 * c);
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
          p.part_ml[part * 2 * kRows + row] = m;
          p.part_ml[(part * 2 + 1) * kRows + row] = l;
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
  return launch_paged<D, kRows>(paged_prefill_kernel<D>, a, L::kPerSm, L::kThreads, L::kSmem, num_sms, stream);
}

}  // namespace

cudaError_t launch_paged_prefill(const PagedAttnArgs& a, int num_sms, cudaStream_t stream) {
  return a.D == 128 ? launch<128>(a, num_sms, stream) : launch<64>(a, num_sms, stream);
}

}  // namespace smla
