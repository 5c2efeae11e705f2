// The matrix product of the MXFP8 operators: W [rows, K] times x [T, K]^T, both
// e4m3 codes with a power-of-two scale per 32 values, as the tensor cores take
// them (tcgen05 kind::mxf8f6f4 with a scale vector: exact products, scaled and
// summed in float32 in tensor memory).
//
// Features are the MMA's rows and tokens its columns (M = 128, N = kNT), so that
// one token costs a tile of 16 columns and not of 128 rows, and so that the 32
// values under one output scale are the 32 lanes of a warp.  A gated product
// holds two accumulators of the same lanes, its gate's and its up part's rows.
//
// A CTA makes one output tile, over all of K or, where tiles are few, over one of
// the equal parts of K that a cluster's CTAs share; each then leaves its partial
// sums in its shared memory and sums up some of the columns, in the order of the
// ranks.  Warp roles: 0 TMA producer (codes, 128-byte rows and swizzle), 1 MMA
// issuer, 2..5 first copy the scale bytes into shared memory in the order in
// which tcgen05.cp takes them to tensor memory (row r's 4 bytes of a 128-value
// step at 16 (r % 32) + 4 (r / 32)), then write the results out.
#pragma once
#include <algorithm>
#include <cstdint>
#include <mutex>
#include <type_traits>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/smla.h"
#include "sm103_ptx.cuh"
#include "smla_common.cuh"
#include "smla_kernels.h"
#include "smla_mxfp8.cuh"

namespace smla {

namespace {

constexpr uint32_t kAllLanes = 0xffffffffu;
constexpr int kStepK = 128;    // values of K per stage: one 128-byte swizzle row
constexpr int kTileRows = 128; // features per accumulator
constexpr int kMxThreads = 6 * 32;

// Set when a wait runs out in a kernel of the file that includes this.
__device__ int g_mx_timed_out;

enum MxMode { kLinear, kMoeUp, kMoeDown };

// ---------------------------------------------------------------- instructions

// Instruction descriptor of kind::mxf8f6f4: e4m3 times e4m3, both K-major, scales
// as exponent bytes; sf: which of the 4 bytes of the scales' columns.
__host__ __device__ constexpr uint32_t idesc_mx(uint32_t M, uint32_t N, uint32_t sf) {
  return (sf << 4) | ((N >> 3) << 17) | (1u << 23) | ((M >> 4) << 24) | (sf << 29);
}
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// 512 bytes of shared memory (32 rows of 16) into 4 columns of tensor memory, the
// same in each quarter of its lanes.  In order with the MMAs of the same thread.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// ---------------------------------------------------------------- parameters and layout

struct MxParams {
  const uint8_t* a_scale;  // of W's rows
  int64_t a_scale_stride;
  const uint8_t* b_scale;  // of the tokens' rows
  int64_t b_scale_stride;
  int rows;                // features (of a gated product: the gate's; the up part's rows follow them)
  int T, K;                // tokens; values of a row
  MxEpilogue to;
  int64_t ld;              // features of an output row
  bool pairs;              // bf16 results and residual can be accessed two at a time
  // mixture of experts
  const int32_t* ids;      // [T, topk]
  const float* weights;
  int topk, E;
  int slots;               // experts that a token tile can have at most
};

template <int NA, int NT>
struct MxLay {
  static constexpr int kATile = kTileRows * kStepK;
  static constexpr int kBTile = NT * kStepK;
  static constexpr int kStage = NA * kATile + kBTile;
  static constexpr int kNB = (NT + 127) / 128;  // 128-row blocks of the tokens' scales
  static constexpr int kScales = 512 * (NA + kNB);
  static constexpr int kMisc = 4096;            // barriers, expert lists, weights
  static constexpr int kBudget = 113 * 1024 - 1024 - kMisc;  // two CTAs an SM
  static constexpr int kFit = kBudget / (kStage + kScales);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kPartial = NA * NT * kTileRows * 4;
  static constexpr int kRing = kStages * kStage > kPartial ? kStages * kStage : kPartial;
  static constexpr int kOffScales = kRing;
  static constexpr int kOffMisc = kOffScales + kStages * kScales;
  static constexpr int kSmem = kOffMisc + kMisc + 1024;
  static constexpr int kAcc = NA * NT;          // tensor memory: accumulators, then two sets of scales
  static constexpr int kScaleCols = 4 * (NA + kNB);
  static constexpr int kNeed = kAcc + 2 * kScaleCols;
  static constexpr int kCols = kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
  static_assert(kStages >= 2 && kStage % 1024 == 0, "stages");
  static_assert(kNeed <= 512 && kSmem <= 232448, "limits");
};

constexpr int kMaxMoeExperts = 1024;
struct MxMisc {
  uint64_t full[6], empty[6], done;
  uint32_t tmem;
  int abort_flag, active;
  uint32_t mask[kMaxMoeExperts / 32];
  uint16_t list[kMaxMoeExperts];
  float share[256];
  uint8_t routed[256];
};
static_assert(sizeof(MxMisc) <= 4096, "misc");

// ---------------------------------------------------------------- the results' way out

__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.f + __expf(-x)); }

__device__ __forceinline__ float activate(int kind, float x) {
  switch (kind) {
    case SMLA_ACT_RELU: return x < 0.f ? 0.f : x;  // (a NaN stays)
    case SMLA_ACT_SILU: return silu(x);
    case SMLA_ACT_GELU: return 0.5f * x * (1.f + erff(x * 0.70710678118654752f));
    // x (1 + tanh u) / 2 = x / (1 + e^(-2 u))
    case SMLA_ACT_GELU_TANH: return __fdividef(x, 1.f + __expf(-1.5957691216057308f * fmaf(0.044715f * x * x, x, x)));
    default: return x;
  }
}
__device__ __forceinline__ float bias_at(const MxEpilogue& to, int64_t i) {
  return to.bias_f32 ? __ldg(static_cast<const float*>(to.bias) + i)
                     : __bfloat162float(static_cast<const __nv_bfloat16*>(to.bias)[i]);
}

// Where results go: MXFP8 codes, bf16 two features an access, bf16 one at a time.
enum MxOut { kOutCodes, kOutPairs, kOutSingle };
__device__ __forceinline__ MxOut out_kind(const MxParams& p) {
  return p.to.out == nullptr ? kOutCodes : p.pairs ? kOutPairs : kOutSingle;
}

// Four tokens' results of this lane's feature f; the lanes of the warp hold 32
// consecutive features from `group` on.  They go to rows out_row .. of the output,
// the first n of them.
template <MxOut kOut>
__device__ __forceinline__ void write_out(const MxParams& p, float (&v)[4], int f, int group, int64_t out_row, int n) {
  const MxEpilogue& to = p.to;
  const int lane = threadIdx.x & 31;
  if (kOut == kOutCodes) {
    // N is a multiple of 32, so the warp's group is whole or not there
    if (group >= p.rows) return;
    int e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[i] = mx_exponent(__reduce_max_sync(kAllLanes, mx_finite_bits(v[i])));
      v[i] *= mx_pow2(-e[i]);
    }
    // bytes: this feature's 4 tokens; exchanged in fours of lanes for one token's 4 features
    uint32_t w = mx_e4m3x4(v[0], v[1], v[2], v[3]);
    uint32_t o = __shfl_xor_sync(kAllLanes, w, 1);
    w = __byte_perm(w, o, lane & 1 ? 0x3715 : 0x6240);
    o = __shfl_xor_sync(kAllLanes, w, 2);
    w = __byte_perm(w, o, lane & 2 ? 0x3276 : 0x5410);
    const int i = lane & 3;
    if (i < n) {
      *reinterpret_cast<uint32_t*>(to.codes + (out_row + i) * p.ld + group + (lane & 28)) = w;
      const int mine = i == 0 ? e[0] : i == 1 ? e[1] : i == 2 ? e[2] : e[3];
      if (lane < 4) to.scales[(out_row + i) * to.scale_stride + group / kMxGroup] = (uint8_t)(mine + 127);
    }
    return;
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(to.out);
  const __nv_bfloat16* res = static_cast<const __nv_bfloat16*>(to.residual);
  if (kOut == kOutPairs) {
    // two features of one token a lane: even lanes take the even token of a pair
    const int even = f & ~1;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const bool odd = lane & 1;
      const float got = __shfl_xor_sync(kAllLanes, odd ? v[i] : v[i + 1], 1);
      float lo = odd ? got : v[i], hi = odd ? v[i + 1] : got;
      const int k = i + (lane & 1);
      if (k >= n || even >= p.rows) continue;
      if (res) {
        const uint32_t r = __ldg(reinterpret_cast<const uint32_t*>(res + (out_row + k) * to.residual_stride + even));
        lo += __uint_as_float(r << 16);
        hi += __uint_as_float(r & 0xffff0000u);
      }
      *reinterpret_cast<uint32_t*>(out + (out_row + k) * p.ld + even) = pack_bf16x2(lo, hi);
    }
    return;
  }
  if (f >= p.rows) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= n) break;
    if (res) v[i] += __bfloat162float(res[(out_row + i) * to.residual_stride + f]);
    out[(out_row + i) * p.ld + f] = __float2bfloat16_rn(v[i]);
  }
}
__device__ __forceinline__ void write_out(MxOut kind, const MxParams& p, float (&v)[4], int f, int group, int64_t out_row,
                                          int n) {
  if (kind == kOutCodes) write_out<kOutCodes>(p, v, f, group, out_row, n);
  else if (kind == kOutPairs) write_out<kOutPairs>(p, v, f, group, out_row, n);
  else write_out<kOutSingle>(p, v, f, group, out_row, n);
}

// ---------------------------------------------------------------- the kernel

// grid: x = cluster rank + parts * row tile, y = token tile, z = expert slot (kMoeUp).
template <int MODE, int NA, int NT>
__global__ void __launch_bounds__(kMxThreads, 2)
    mx_gemm_kernel(const __grid_constant__ MxParams p, const int parts, const __grid_constant__ CUtensorMap a_map,
                   const __grid_constant__ CUtensorMap b_map) {
  using L = MxLay<NA, NT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  MxMisc& m = *reinterpret_cast<MxMisc*>(smem + L::kOffMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)blockIdx.x % parts, n0 = (int)blockIdx.x / parts * kTileRows;
  const int t0 = (int)blockIdx.y * NT, ntok = min(NT, p.T - t0);
  volatile int* abort_flag = &m.abort_flag;

  if (tid == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&m.full[s], 5);  // the producer and four warps' scales
      mbar_init(&m.empty[s], 1);
    }
    mbar_init(&m.done, 1);
    m.abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(&m.tmem, L::kCols);
    tmem_relinquish();
  }
  if (MODE != kLinear && tid < kMaxMoeExperts / 32) m.mask[tid] = 0u;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m.tmem;

  // What precedes on the stream is complete behind this.  The experts' second
  // product is launched while the first runs: its choice of experts and its
  // weights were there before that, and only what the first writes is waited for, below.
  if (MODE != kMoeDown) grid_dependency_wait();
  if (MODE == kMoeUp) grid_launch_dependents();

  const int steps = (p.K + kStepK - 1) / kStepK;  // of one row
  int total = steps, expert = 0, active = 1;
  if (MODE != kLinear) {
    // the experts that this tile's tokens go to, in order
    for (int i = tid; i < ntok * p.topk; i += kMxThreads) {
      const int id = __ldg(p.ids + (int64_t)t0 * p.topk + i);
      if (id >= 0 && id < p.E) atomicOr(&m.mask[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
    if (tid < 32) {
      const uint32_t word = m.mask[lane];
      int before = __popc(word);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAllLanes, before, d);
        if (lane >= d) before += o;
      }
      int at = before - __popc(word);
      for (uint32_t w = word; w; w &= w - 1) m.list[at++] = (uint16_t)(32 * lane + __ffs(w) - 1);
      if (lane == 31) m.active = before;
    }
    __syncthreads();
    active = m.active;
    if (MODE == kMoeUp) {
      const bool idle = (int)blockIdx.z >= active;  // the same for a whole cluster
      expert = idle ? 0 : m.list[blockIdx.z];
      if (idle) total = 0;
      // the weight that each token gives this expert
      for (int t = tid; t < NT; t += kMxThreads) {
        float w = 0.f;
        bool any = false;
        if (t < ntok)
          for (int k = 0; k < p.topk; ++k) {
            const int64_t i = (int64_t)(t0 + t) * p.topk + k;
            if (__ldg(p.ids + i) == expert) w += __ldg(p.weights + i), any = true;
          }
        m.share[t] = w;
        m.routed[t] = any;
      }
      __syncthreads();
    } else {
      total = active * steps;
    }
  }
  const int k0 = (int)((int64_t)total * rank / parts), n = (int)((int64_t)total * (rank + 1) / parts) - k0;
  const int slot0 = MODE == kMoeUp ? (int)(blockIdx.y * p.slots + blockIdx.z) : (int)blockIdx.y * p.slots;

#define MX_WAIT(bar, parity) mbar_wait(&(bar), (parity), abort_flag, &g_mx_timed_out, kDevWaitTimeout)
  bool dead = false;
  if (warp == 0) {
    // ---------------------------------------------------------------- codes
    if (lane == 0) {
      auto load_a = [&](int i) {
        const int s = i % L::kStages, it = k0 + i;
        const uint32_t stage = smem_u32(smem + s * L::kStage);
        const int x = (MODE == kMoeDown ? it % steps : it) * kStepK;
        const int e = MODE == kMoeUp ? expert : MODE == kMoeDown ? m.list[it / steps] : 0;
        const int y = e * NA * p.rows + n0;
        mbar_arrive_expect_tx(&m.full[s], (uint32_t)L::kStage);
        tma_load_2d(stage, &a_map, x, y, &m.full[s]);
        if (NA == 2) tma_load_2d(stage + L::kATile, &a_map, x, y + p.rows, &m.full[s]);
      };
      auto load_b = [&](int i) {
        const int s = i % L::kStages, it = k0 + i;
        const int x = (MODE == kMoeDown ? it % steps : it) * kStepK;
        const int y = MODE == kMoeDown ? (slot0 + it / steps) * NT : t0;
        tma_load_2d(smem_u32(smem + s * L::kStage) + NA * L::kATile, &b_map, x, y, &m.full[s]);
      };
      const int early = MODE == kMoeDown ? min(n, L::kStages) : 0;
      for (int i = 0; i < early; ++i) load_a(i);
      if (MODE == kMoeDown) grid_dependency_wait();
      for (int i = 0; i < early; ++i) load_b(i);
      int issued = early;
      for (int i = early; i < n; ++i) {
        if (i >= L::kStages && !MX_WAIT(m.empty[i % L::kStages], ((i / L::kStages) + 1) & 1)) break;
        load_a(i);
        load_b(i);
        ++issued;
      }
      // no copy may still be landing when the CTA exits (after an abort: the last of each stage)
      if (*abort_flag)
        for (int i = max(0, issued - L::kStages); i < issued; ++i)
          mbar_wait_drain(&m.full[i % L::kStages], (i / L::kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      for (int i = 0; i < n; ++i) {
        const int s = i % L::kStages;
        if (!MX_WAIT(m.full[s], (i / L::kStages) & 1)) break;
        tc_fence_after();
        const uint32_t stage = smem_u32(smem + s * L::kStage), scales = smem_u32(smem + L::kOffScales + s * L::kScales);
        const uint32_t sf = tmem + L::kAcc + (i & 1) * L::kScaleCols;
#pragma unroll
        for (int j = 0; j < NA + L::kNB; ++j)
          tmem_copy_scales(sf + 4 * j, make_sdesc(scales + 512 * j, 16, 128, kLayoutNone));
#pragma unroll
        for (int k = 0; k < kStepK / 32; ++k)
#pragma unroll
          for (int a = 0; a < NA; ++a)
            mma_mx(tmem + a * NT, make_sdesc(stage + a * L::kATile + 32 * k, 16, 1024, kLayoutSw128),
                   make_sdesc(stage + NA * L::kATile + 32 * k, 16, 1024, kLayoutSw128), idesc_mx(kTileRows, NT, k),
                   sf + 4 * a, sf + 4 * NA, (i > 0 || k > 0) ? 1u : 0u);
        mma_commit(&m.empty[s]);
      }
      mma_commit(&m.done);
      mbar_wait_drain(&m.done, 0);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- scales
    if (MODE == kMoeDown) grid_dependency_wait();
    const int q = warp & 3, r = 32 * q + lane;
    constexpr int kAhead = 4, kWords = NA + L::kNB;
    const int groups = p.K / kMxGroup;
    auto load = [&](int i, uint32_t (&w)[kWords]) {
      const int it = k0 + i, x = MODE == kMoeDown ? it % steps : it;
      const int e = MODE == kMoeUp ? expert : MODE == kMoeDown ? m.list[it / steps] : 0;
      const int left = groups - 4 * x;  // bytes of the row's last word behind its end count for nothing
      const uint32_t valid = left >= 4 ? ~0u : (1u << (8 * left)) - 1u;
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        const int64_t row = ((int64_t)e * NA + a) * p.rows + n0 + r;
        w[a] = n0 + r < p.rows
                   ? __ldg(reinterpret_cast<const uint32_t*>(p.a_scale + row * p.a_scale_stride + 4 * x)) & valid
                   : 0u;
      }
#pragma unroll
      for (int b = 0; b < L::kNB; ++b) {
        const int c = 128 * b + r;
        const int64_t row = MODE == kMoeDown ? (int64_t)(slot0 + it / steps) * NT + c : t0 + c;
        w[NA + b] = c < ntok
                        ? __ldg(reinterpret_cast<const uint32_t*>(p.b_scale + row * p.b_scale_stride + 4 * x)) & valid
                        : 0u;
      }
    };
    uint32_t cur[kAhead][kWords], nxt[kAhead][kWords];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (j < n) load(j, nxt[j]);
    for (int i0 = 0; i0 < n && !dead; i0 += kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
#pragma unroll
        for (int w = 0; w < kWords; ++w) cur[j][w] = nxt[j][w];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i0 + kAhead + j < n) load(i0 + kAhead + j, nxt[j]);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = i0 + j, s = i % L::kStages;
        if (i >= n || dead) break;
        if (i >= L::kStages)
          dead = __any_sync(kAllLanes, !MX_WAIT(m.empty[s], ((i / L::kStages) + 1) & 1));
        if (dead) break;
        const uint32_t to = smem_u32(smem + L::kOffScales + s * L::kScales) + 16 * lane + 4 * q;
#pragma unroll
        for (int w = 0; w < kWords; ++w)
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + 512 * w), "r"(cur[j][w]) : "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.full[s]);
      }
    }
    dead = __any_sync(kAllLanes, dead || !MX_WAIT(m.done, 0));
    tc_fence_after();
  }

  // ---------------------------------------------------------------- results
  const int q = warp & 3, f = n0 + 32 * q + lane;
  const MxOut out = out_kind(p);
  float bias[NA];
  if (warp >= 2)
#pragma unroll
    for (int a = 0; a < NA; ++a)
      bias[a] = MODE == kLinear && p.to.bias && f < p.rows ? bias_at(p.to, (int64_t)a * p.rows + f) : 0.f;
  auto finish = [&](float (&v)[NA][4], int c) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = v[0][i] + bias[0];
      if (NA == 2) y[i] = silu(y[i]) * (v[NA - 1][i] + bias[NA - 1]);
      else if (MODE == kLinear) y[i] = activate(p.to.activation, y[i]);
      if (MODE == kMoeUp) y[i] = c + i < ntok && m.routed[c + i] ? y[i] * m.share[c + i] : 0.f;
    }
    const int64_t row = MODE == kMoeUp ? (int64_t)slot0 * NT + c : t0 + c;
    write_out(out, p, y, f, n0 + 32 * q, row, ntok - c);
  };
  const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16);
  if (MODE == kMoeUp && total == 0) {
    // no such expert: nothing to compute, nothing to write
  } else if (parts == 1) {
    if (warp >= 2 && !dead) {
#pragma unroll 1
      for (int c = 0; c < ntok; c += 8) {
        uint32_t w[NA][8];
#pragma unroll
        for (int a = 0; a < NA; ++a) tmem_ld8(acc + a * NT + c, w[a]);
        tmem_ld_wait();
#pragma unroll
        for (int a = 0; a < NA; ++a) reg_fence8(w[a]);
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
          float v[NA][4];
#pragma unroll
          for (int a = 0; a < NA; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[a][i] = n > 0 ? __uint_as_float(w[a][h + i]) : 0.f;
          if (c + h < ntok) finish(v, c + h);
        }
      }
    }
  } else {
    float* part = reinterpret_cast<float*>(smem);  // [accumulator][column][row]; every copy and MMA has ended
    if (warp >= 2) {
#pragma unroll 1
      for (int c = 0; c < ntok; c += 8) {
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          uint32_t w[8];
          tmem_ld8(acc + a * NT + c, w);
          tmem_ld_wait();
          reg_fence8(w);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            part[(a * NT + c + i) * kTileRows + 32 * q + lane] = n > 0 ? __uint_as_float(w[i]) : 0.f;
        }
      }
    }
    __syncwarp();
    cluster_sync_all();
    if (warp >= 2 && !dead) {
      const uint32_t mine = smem_u32(part) + 4 * (32 * q + lane);
#pragma unroll 1
      for (int c = 4 * rank; c < ntok; c += 4 * parts) {
        float v[NA][4] = {};
        for (int o = 0; o < parts; ++o) {
          const uint32_t from = mapa_shared(mine, (uint32_t)o);
#pragma unroll
          for (int a = 0; a < NA; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[a][i] += ld_cluster_f32(from + 4 * kTileRows * (a * NT + c + i));
        }
        finish(v, c);
      }
    }
    __syncwarp();
    cluster_sync_relaxed();  // no CTA leaves while another reads its sums
  }
#undef MX_WAIT
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

// ---------------------------------------------------------------- launch

using MxEncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

MxEncodeFn mx_encode_fn() {
  static MxEncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<MxEncodeFn>(ptr);
  });
  return fn;
}

// Bytes [rows, cols], rows `stride` bytes apart (a multiple of 16), in boxes; what
// lies outside reads as zeros.
cudaError_t byte_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t stride, int box_cols,
                     int box_rows, CUtensorMapSwizzle swizzle) {
  MxEncodeFn enc = mx_encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)stride};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, es[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
// Codes [rows, K] in boxes of 128 bytes of box_rows rows.
cudaError_t code_map(CUtensorMap* map, const void* base, int64_t rows, int64_t K, int64_t stride, int box_rows) {
  return byte_map(map, base, rows, K, stride, kStepK, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int MODE, int NA, int NT>
cudaError_t launch_mx(const MxParams& p, int parts, int64_t row_tiles, int64_t token_tiles, int slots,
                      const CUtensorMap& a_map, const CUtensorMap& b_map, cudaStream_t stream) {
  if (row_tiles * parts > INT32_MAX || token_tiles > 65535 || slots > 65535) return cudaErrorInvalidValue;
  auto kernel = mx_gemm_kernel<MODE, NA, NT>;
  constexpr int smem = MxLay<NA, NT>::kSmem;
  // at every launch: it takes well under a microsecond and needs no per-device record
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(row_tiles * parts), (unsigned)token_tiles, (unsigned)slots);
  cfg.blockDim = dim3(kMxThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p, parts, a_map, b_map);
}

// Parts of K: as many as give every SM two CTAs, each with two steps or more.
int split_k(int64_t tiles, int64_t steps, int num_sms) {
  int parts = 1;
  while (parts < 8 && tiles * parts * 2 <= 2 * (int64_t)num_sms && steps >= 4 * parts) parts *= 2;
  return parts;
}

}  // namespace

}  // namespace smla
