// The same product for many tokens: tiles of 256 features by 256 tokens (gated:
// 256 by 128, gate and up part) by pairs of CTAs, whose MMAs (cta_group::2,
// M = 256) read each CTA's 128 features from its own shared memory and half of the
// tokens from each, so that an SM loads and reads half the tokens' bytes.  The
// pairs are persistent; a tile's accumulator (256 columns) is emptied into
// registers at once, and while its results are written the next tile's MMAs run.
//
// Scales: rows of 32 bytes (8 steps of K) of the tile's 384 scale rows come by TMA
// (where they lie on 16-byte boundaries, otherwise word by word);
// four warps, one for each quarter of the lanes of tensor memory, store them there,
// four steps at a time.  (Through shared memory and tcgen05.cp, the copies stood
// between the MMAs: 2501 x 5120 x 13824 took 166 us where it took 140 without any
// scales.)  What one CTA tells the other
// by an arrival lies in tensor memory or has been read, not in memory: the arrivals
// are relaxed.  (One that releases at cluster scope waits for the SM's stores in
// flight: 301 us against 153.)
//
// Warp roles: 0 TMA of the codes (each CTA loads its halves, both count on the
// first one's barriers), 1 MMA issuer (in the first CTA), 2 TMA of the scales,
// 4..7 scales, 8..15 results.
//
// Measured, alone and (at the power limit, 1.4 kW) in a row: 2501 x 5120 x 13824
// with gelu 114 and 134 us (3.1 and 2.6 PFLOP/s), 6000 x 4096 x 2 * 8192 gated to
// MXFP8 238 and 282 us (3.4 and 2.9); the MMAs alone, without copies and results,
// take 91 and 179.  Between them and the whole lie the switch of a tile (the
// accumulator of 256 columns has no second place beside the scales), results that
// share tensor memory and issue slots with the MMAs, and with few turns of tiles
// the last one.  Copies of the features' codes shared by two pairs (multicast in a
// cluster of four, of which 144 SMs hold some) were slower, 2501 x 5120 x 13824 in 376
// us where it took 343 then; so was asking for them early, into L2, 148 against 137.
#pragma once
#include "smla_mxgemm.cuh"

namespace smla {

namespace {

// ---------------------------------------------------------------- instructions

__device__ __forceinline__ void pair_alloc(uint32_t* slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this place in both CTAs when all MMAs so far have completed.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// tma_load_2d into this CTA, counted on a barrier of either CTA of the pair (cluster address).
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const void* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// True in the four warps of the scales if it is in any of their threads.
__device__ __forceinline__ bool scale_warps_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// ---------------------------------------------------------------- layout

constexpr int kPairSets = 4;

template <int NA>
struct PairLay {
  static constexpr int kTokens = 256 / NA;             // of a tile: the accumulator's 256 columns
  static constexpr int kBTile = kTokens / 2 * kStepK;  // a CTA's half of the tokens
  static constexpr int kStage = NA * kTileRows * kStepK + kBTile;
  static constexpr int kBlocks = NA + kTokens / 128;   // of 128 scale rows: of the features, then of the tokens
  static constexpr int kStages = NA == 1 ? 6 : 5;
  static constexpr int kRawBlock = 128 * 32, kRaw = kBlocks * kRawBlock;
  static constexpr int kOffRaw = kStages * kStage;
  static constexpr int kOffMisc = kOffRaw + 2 * kRaw;
  static constexpr int kSmem = kOffMisc + 256 + 1024;
  static constexpr int kAcc = 256, kScaleCols = 4 * kBlocks;  // of a step; four steps make a set, kPairSets of them a ring
  static constexpr int kCols = 512;
  static_assert(kSmem <= 232448 && kStage % 1024 == 0 && kAcc + kPairSets * 4 * kScaleCols <= kCols, "limits");
};
struct PairMisc {
  uint64_t full[6], empty[6], scaled[kPairSets], unscaled[kPairSets], raw_full[2], raw_empty[2], acc_full, acc_empty, idle;
  uint32_t tmem;
  int abort_flag;
  int codes, scales;  // copies that this CTA has issued: of codes (a stage each), of scales (a buffer each)
};
static_assert(sizeof(PairMisc) <= 256, "misc");

constexpr int kPairThreads = 512;
// Registers a thread by warpgroup, of 128 at launch: 64 + 96 + 2 * 176 = 4 * 128.
constexpr int kRoleRegs = 64, kScaleRegs = 96, kResultRegs = 176;

// ---------------------------------------------------------------- the kernel

template <int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    mx_pair_kernel(const __grid_constant__ MxParams p, const int whole, const int cut, const __grid_constant__ CUtensorMap a_map,
                   const __grid_constant__ CUtensorMap b_map, const __grid_constant__ CUtensorMap a_scale_map,
                   const __grid_constant__ CUtensorMap b_scale_map) {
  constexpr int NA = ACT == SMLA_ACT_SWIGLU ? 2 : 1;
  using L = PairLay<NA>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  PairMisc& m = *reinterpret_cast<PairMisc*>(smem + L::kOffMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank();
  volatile int* abort_flag = &m.abort_flag;

  if (tid == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&m.full[s], 1);
      mbar_init(&m.empty[s], 1);
    }
    for (int b = 0; b < kPairSets; ++b) {
      mbar_init(&m.scaled[b], 8);  // four warps in each CTA
      mbar_init(&m.unscaled[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&m.raw_full[b], 1);
      mbar_init(&m.raw_empty[b], 4);
    }
    mbar_init(&m.acc_full, 1);
    mbar_init(&m.acc_empty, 16);
    mbar_init(&m.idle, 1);
    m.abort_flag = p.give_up;
    m.codes = m.scales = 0;
    mbar_fence_init();
  }
  if (warp == 1) pair_alloc(&m.tmem, L::kCols);
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = m.tmem;
  grid_dependency_wait();

  const int steps = (p.K + kStepK - 1) / kStepK;
  const int token_tiles = (p.T + L::kTokens - 1) / L::kTokens, row_tiles = (p.rows + 2 * kTileRows - 1) / (2 * kTileRows);
  // Units: the whole tiles, then those that are cut into `cut` parts of fewer tokens.
  const int first = (int)blockIdx.x / 2, stride = (int)gridDim.x / 2;
  struct Unit {
    int row, token, tokens;  // this CTA's first feature; the first token and how many columns
  };
  auto unit_at = [&](int u) {
    const int v = u - whole, tile = v < 0 ? u : whole + v / cut;
    Unit x;
    x.row = tile / token_tiles * (2 * kTileRows) + rank * kTileRows;
    x.tokens = v < 0 ? L::kTokens : L::kTokens / cut;
    x.token = tile % token_tiles * L::kTokens + (v < 0 ? 0 : v % cut * x.tokens);
    return x;
  };
  const int units = whole + (token_tiles * row_tiles - whole) * cut;
  // The next unit that has tokens, from u on.
  auto next_unit = [&](int u, Unit& x) {
    for (; u < units; u += stride) {
      x = unit_at(u);
      if (x.token < p.T) break;
    }
    return u;
  };

#define PAIR_WAIT(bar, parity) mbar_wait(&(bar), (parity), abort_flag, &g_mx_timed_out, kDevWaitTimeout)
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------------- codes
      int i = 0;
      bool ok = true;
      Unit x;
      for (int u = next_unit(first, x); u < units && ok; u = next_unit(u + stride, x)) {
        const int y = x.row, t = x.token + rank * (x.tokens / 2);
        for (int k = 0; k < steps; ++k, ++i) {
          const int s = i % L::kStages, use = i / L::kStages;
          if (use > 0 && !(ok = PAIR_WAIT(m.empty[s], (use + 1) & 1))) break;
          const uint32_t stage = smem_u32(smem + s * L::kStage), bar = mapa_shared(smem_u32(&m.full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&m.full[s], 2u * L::kStage);
#pragma unroll
          for (int a = 0; a < NA; ++a)
            pair_load_2d(stage + a * kTileRows * kStepK, &a_map, k * kStepK, y + a * p.rows, bar);
          pair_load_2d(stage + NA * kTileRows * kStepK, &b_map, k * kStepK, t, bar);
        }
      }
      m.codes = i;
    } else if (warp == 1 && rank == 0) {
      // -------------------------------------------------------------- MMA issuer
      // The whole warp goes through the loop and elects the issuing thread at each step, so that the operands lie in
      // uniform registers; descriptors differ by one addition.  (One thread's loop, with descriptors made anew, was what
      // bound the kernel: 155 us instead of 122.)
      constexpr uint32_t kHi = sdesc_hi(1024, kLayoutSw128);
      const uint32_t lo0 = sdesc_lo(smem_u32(smem), 16);
      int s = 0, set = 0, n = 0;
      uint32_t phase = 0, set_phase = 0;
      bool ok = true;
      Unit x;
      for (int u = next_unit(first, x); u < units && ok; u = next_unit(u + stride, x), ++n) {
        if (n > 0 && !(ok = PAIR_WAIT(m.acc_empty, (n + 1) & 1))) break;
        tc_fence_after();
        const uint32_t idesc = idesc_mx(2 * kTileRows, (uint32_t)x.tokens, 0);
        for (int k0 = 0; k0 < steps && ok; k0 += 4) {
          if (!(ok = PAIR_WAIT(m.scaled[set], set_phase))) break;
          const int left = min(4, steps - k0);
          uint32_t sf = tmem + L::kAcc + 4 * set * L::kScaleCols;
          for (int k = 0; k < left; ++k, sf += L::kScaleCols) {
            if (!(ok = PAIR_WAIT(m.full[s], phase))) break;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t lo = lo0 + (uint32_t)s * (L::kStage >> 4);
#pragma unroll
              for (int kk = 0; kk < kStepK / 32; ++kk)
#pragma unroll
                for (int a = 0; a < NA; ++a)
                  pair_mma(tmem + a * L::kTokens, sdesc_join<kHi>(lo + ((a * kTileRows * kStepK + 32 * kk) >> 4)),
                           sdesc_join<kHi>(lo + ((NA * kTileRows * kStepK + 32 * kk) >> 4)),
                           idesc | idesc_sf(kk), sf + 4 * a, sf + 4 * NA,
                           kk > 0 ? 1u : (uint32_t)((k0 | k) != 0));
              pair_commit(&m.empty[s]);
              if (k + 1 == left) pair_commit(&m.unscaled[set]);
              if (k0 + k + 1 == steps) pair_commit(&m.acc_full);
            }
            __syncwarp();
            if (++s == L::kStages) s = 0, phase ^= 1;
          }
          if (++set == kPairSets) set = 0, set_phase ^= 1;
        }
      }
    } else if (warp == 2 && lane == 0 && p.wide_scales) {
      // -------------------------------------------------------------- scales' bytes
      int i = 0;
      bool ok = true;
      Unit x;
      for (int u = next_unit(first, x); u < units && ok; u = next_unit(u + stride, x)) {
        const int y = x.row, t = x.token;
        for (int k = 0; k < steps; k += 8, ++i) {
          const int b = i & 1;
          if (i >= 2 && !(ok = PAIR_WAIT(m.raw_empty[b], ((i >> 1) + 1) & 1))) break;
          const uint32_t raw = smem_u32(smem + L::kOffRaw + b * L::kRaw);
          mbar_arrive_expect_tx(&m.raw_full[b], (uint32_t)L::kRaw);
#pragma unroll
          for (int j = 0; j < L::kBlocks; ++j)
            tma_load_2d(raw + j * L::kRawBlock, j < NA ? &a_scale_map : &b_scale_map, 4 * k,
                        j < NA ? y + j * p.rows : t + 128 * (j - NA), &m.raw_full[b]);
        }
      }
      m.scales = i;
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---------------------------------------------------------------- scales
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kScaleRegs));
    const uint32_t to = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + L::kAcc;
    // Scale rows that TMA cannot copy: thread t copies word by word the t-th row of each block, eight steps ahead.
    const int thread = 32 * (warp - 4) + lane;
    int next_u = 0, next_k = 0, next_b = 0;
    Unit next{};
    auto copy_next = [&]() {
      if (next_u < units) {
        const uint32_t raw = smem_u32(smem + L::kOffRaw + next_b * L::kRaw) + 32 * thread;
#pragma unroll
        for (int j = 0; j < L::kBlocks; ++j) {
          const bool features = j < NA;
          const int at = features ? next.row + thread : next.token + 128 * (j - NA) + thread;
          const bool there = at < (features ? p.rows : p.T);
          const uint8_t* row = features ? p.a_scale + ((int64_t)j * p.rows + at) * p.a_scale_stride
                                        : p.b_scale + (int64_t)at * p.b_scale_stride;
          for (int k = 0; k < 8 && next_k + k < steps; ++k)
            cp_async4_zfill(raw + j * L::kRawBlock + 4 * k, there ? row + 4 * (next_k + k) : p.a_scale,
                            there ? (uint32_t)min(p.K / kMxGroup - 4 * (next_k + k), 4) : 0u);
        }
        next_k += 8;
        if (next_k >= steps) next_k = 0, next_u = next_unit(next_u + stride, next);
      }
      next_b ^= 1;
    };
    if (!p.wide_scales) {
      next_u = next_unit(first, next);
      copy_next();
    }
    int g = 0, r = 0;
    bool dead = false, stop = false;  // (without TMA a warp that gives up goes on to the next meeting with the others)
    Unit x;
    for (int u = next_unit(first, x); u < units && !stop; u = next_unit(u + stride, x)) {
      for (int k = 0; k < steps; k += 4, ++g) {
        const int b = r & 1, set = g % kPairSets, half = k & 4;
        const bool read = half != 0 || k + 4 >= steps;  // the buffer is done with behind this
        if (half == 0 && p.wide_scales) dead = __any_sync(kAllLanes, !PAIR_WAIT(m.raw_full[b], (r >> 1) & 1));
        if (half == 0 && !p.wide_scales) {
          cp_async_commit();
          cp_async_wait<0>();
          stop = scale_warps_any(dead);  // everyone's copies are there, and everyone has read the other buffer
          if (stop) break;
          copy_next();
        }
        if (!dead && g >= kPairSets) dead = __any_sync(kAllLanes, !PAIR_WAIT(m.unscaled[set], (g / kPairSets + 1) & 1));
        if (dead) {
          stop = p.wide_scales;
          if (stop) break;
          r += read;
          continue;
        }
        tc_fence_after();
        // lane l: four steps' words of rows l, l + 32, l + 64, l + 96 of each block; column 4 j + c of a step is block j's c-th
        uint4 w[L::kBlocks][4];
#pragma unroll
        for (int j = 0; j < L::kBlocks; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            w[j][c] = *reinterpret_cast<const uint4*>(smem + L::kOffRaw + b * L::kRaw + j * L::kRawBlock + (32 * c + lane) * 32 +
                                                      4 * half);
        uint32_t v[4 * L::kScaleCols];
#pragma unroll
        for (int j = 0; j < L::kBlocks; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4& u = w[j][c];
            v[4 * j + c] = u.x;
            v[L::kScaleCols + 4 * j + c] = u.y;
            v[2 * L::kScaleCols + 4 * j + c] = u.z;
            v[3 * L::kScaleCols + 4 * j + c] = u.w;
          }
        static_assert(L::kScaleCols == 12, "48 columns");
#pragma unroll
        for (int c = 0; c < 48; c += 16)
          tmem_st16(to + 4 * set * L::kScaleCols + c, *reinterpret_cast<const uint32_t(*)[16]>(v + c));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&m.scaled[set]), 0));
          if (read && p.wide_scales) mbar_arrive(&m.raw_empty[b]);
        }
        r += read;
      }
    }
    cp_async_wait<0>();
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- results
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kResultRegs));
    const int q = warp & 3, half = (warp - 8) >> 2;
    constexpr int kMine = L::kTokens / 2;  // tokens of this warp, at most
    const uint32_t empty = mapa_shared(smem_u32(&m.acc_empty), 0);
    const MxOut kind = out_kind(p);
    int n = 0;
    Unit x;
    for (int u = next_unit(first, x); u < units; u = next_unit(u + stride, x), ++n) {
      const int group = x.row + 32 * q, f = group + lane, t = x.token + half * (x.tokens / 2);
      const int ntok = min(p.T - t, x.tokens / 2);
      const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + half * (x.tokens / 2);
      float bias[NA];
#pragma unroll
      for (int a = 0; a < NA; ++a) bias[a] = p.to.bias && f < p.rows ? bias_at(p.to, (int64_t)a * p.rows + f) : 0.f;
      if (__any_sync(kAllLanes, !PAIR_WAIT(m.acc_full, n & 1))) break;
      tc_fence_after();
      uint32_t w[NA * kMine];
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int c = 0; c < kMine; c += 32) tmem_ld32(acc + a * L::kTokens + c, w + a * kMine + c);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < NA * kMine; ++i) asm volatile("" : "+r"(w[i]));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(empty);
      auto result = [&](int c) {
        const float z = __uint_as_float(w[c]) + bias[0];
        return NA == 2 ? silu(z) * (__uint_as_float(w[(NA - 1) * kMine + c]) + bias[NA - 1])
                       : ACT == SMLA_ACT_GELU ? gelu(z) : activate(ACT, z);
      };
      // 16 tokens at a time without a branch, so that their chains of operations overlap
      constexpr int kAtOnce = 16;
      if (kind == kOutCodes && group < p.rows) {
        uint8_t* codes = p.to.codes + (int64_t)(t + (lane & 3)) * p.ld + group + (lane & 28);
        uint8_t* scales = p.to.scales + (int64_t)(t + (lane & 3)) * p.to.scale_stride + group / kMxGroup;
#pragma unroll
        for (int c0 = 0; c0 < kMine; c0 += kAtOnce) {
          if (c0 >= ntok) break;
#pragma unroll
          for (int c = c0; c < c0 + kAtOnce; c += 4) {
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = result(c + i);
            uint32_t scale;
            const uint32_t v = quantize4(y, scale);
            if (c + (lane & 3) < ntok) {
              *reinterpret_cast<uint32_t*>(codes) = v;
              if (lane < 4) *scales = (uint8_t)scale;
            }
            codes += 4 * p.ld;
            scales += 4 * p.to.scale_stride;
          }
        }
      } else if (kind == kOutPairs) {
        const int64_t row = t + (lane & 1);
        const int even = f & ~1, last = even < p.rows ? ntok : 0;  // this lane's tokens
        uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.to.out) + row * p.ld + even);
        const uint32_t* res = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.to.residual) +
                                                                row * p.to.residual_stride + even);
        auto rows = [&](auto with_residual) {
          constexpr bool kResidual = decltype(with_residual)::value;
#pragma unroll
          for (int c0 = 0; c0 < kMine; c0 += kAtOnce) {
            if (c0 >= ntok) break;
            uint32_t r[kAtOnce / 2];
            if (kResidual) {
#pragma unroll
              for (int i = 0; i < kAtOnce / 2; ++i, res += p.to.residual_stride)  // (plain loads: out may be the residual)
                r[i] = c0 + 2 * i + (lane & 1) < last ? *res : 0u;
            }
#pragma unroll
            for (int i = 0; i < kAtOnce / 2; ++i, out += p.ld) {
              float lo, hi;
              pair_up(result(c0 + 2 * i), result(c0 + 2 * i + 1), lo, hi);
              if (kResidual) {
                lo += __uint_as_float(r[i] << 16);
                hi += __uint_as_float(r[i] & 0xffff0000u);
              }
              if (c0 + 2 * i + (lane & 1) < last) *out = pack_bf16x2(lo, hi);
            }
          }
        };
        if (p.to.residual) rows(std::true_type{});
        else rows(std::false_type{});
      } else if (kind == kOutSingle) {
#pragma unroll
        for (int c = 0; c < kMine; c += 4) {
          if (c >= ntok) break;
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = result(c + i);
          write_out<kOutSingle>(p, y, f, group, t + c, ntok - c);
        }
      }
    }
    if (p.publish) __threadfence();
  }
#undef PAIR_WAIT
  tc_fence_before();
  __syncwarp();
  // Where a wait ran out both CTAs unwind: whose warp raised the flag raises the other CTA's.
  if (lane == 0 && *abort_flag) st_cluster_u32(mapa_shared(smem_u32(&m.abort_flag), (uint32_t)rank ^ 1u), 1u);
  __syncwarp();
  cluster_sync_all();
  if (*abort_flag) {
    // Nothing may be under way any more when the CTAs end: MMAs read both CTAs' memory, copies land in it.
    if (warp == 1) {
      if (rank == 0 && elect_one()) pair_commit(&m.idle);
      __syncwarp();
      mbar_wait_drain(&m.idle, 0);
    } else if (tid == 0 && rank == 0) {
      // both CTAs' copies count on the barriers here, and one may have issued up to kStages more than the other
      const int mine = m.codes, other = (int)ld_cluster_u32(mapa_shared(smem_u32(&m.codes), 1)), most = max(mine, other);
      for (int j = max(0, most - L::kStages); j < most; ++j) {
        const int s = j % L::kStages;
        if (j >= mine) mbar_arrive_expect_tx(&m.full[s], L::kStage);
        if (j >= other) mbar_complete_tx(&m.full[s], L::kStage);
        mbar_wait_drain(&m.full[s], (j / L::kStages) & 1);
      }
    } else if (warp == 2) {
      for (int j = max(0, m.scales - 2); j < m.scales; ++j) mbar_wait_drain(&m.raw_full[j & 1], (j >> 1) & 1);
    }
    if (tid == 0) atomicExch(&g_mx_timed_out, kDevWaitTimeout);
    __syncwarp();
    cluster_sync_all();
  }
  if (warp == 1) {
    tc_fence_after();
    pair_dealloc(tmem, L::kCols);
  }
}

// Scales [rows, n] in boxes of 8 steps' bytes of 128 rows.
cudaError_t scale_map(CUtensorMap* map, const void* base, int64_t rows, int64_t n, int64_t stride) {
  return byte_map(map, base, rows, n, stride, 32, 128, CU_TENSOR_MAP_SWIZZLE_NONE);
}
template <int ACT>
cudaError_t launch_pair(const MxLinearArgs& a, const MxParams& p, int num_sms, cudaStream_t stream) {
  constexpr int NA = ACT == SMLA_ACT_SWIGLU ? 2 : 1;
  using L = PairLay<NA>;
  CUtensorMap a_map, b_map, a_scale_map, b_scale_map;
  cudaError_t e = code_map(&a_map, a.w, (int64_t)NA * a.N, a.K, a.K, kTileRows);
  if (e == cudaSuccess) e = code_map(&b_map, a.x, a.T, a.K, a.x_stride, L::kTokens / 2);
  a_scale_map = b_scale_map = a_map;  // (unused without 16-byte boundaries)
  if (e == cudaSuccess && p.wide_scales)
    e = scale_map(&a_scale_map, a.w_scale, (int64_t)NA * a.N, a.K / kMxGroup, a.w_scale_stride);
  if (e == cudaSuccess && p.wide_scales) e = scale_map(&b_scale_map, a.x_scale, a.T, a.K / kMxGroup, a.x_scale_stride);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (((int64_t)a.T + L::kTokens - 1) / L::kTokens) * (((int64_t)a.N + 2 * kTileRows - 1) / (2 * kTileRows));
  if (tiles > INT32_MAX / 4) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> allowed{0};
  e = allow_smem(mx_pair_kernel<ACT>, L::kSmem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  // The tiles that do not fill the pairs a last time are cut into parts of fewer tokens where that makes a last turn of
  // parts: a turn of half the columns takes 0.6 of the time, of a quarter or an eighth half of it.
  constexpr int kMaxCut = L::kTokens / 32;
  const int64_t pairs = std::max(1, num_sms / 2), left = tiles % pairs;
  int cut = 1;
  while (left > 0 && cut < kMaxCut && left * cut * 2 <= pairs) cut *= 2;
  const int64_t whole = cut > 1 ? tiles - left : tiles, units = whole + (tiles - whole) * cut;
  cfg.gridDim = dim3((unsigned)(2 * std::min(units, pairs)));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mx_pair_kernel<ACT>, p, (int)whole, cut, a_map, b_map, a_scale_map, b_scale_map);
}

}  // namespace

}  // namespace smla
