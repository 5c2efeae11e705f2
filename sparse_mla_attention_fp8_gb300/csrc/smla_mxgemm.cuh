// The matrix product of the MXFP8 operators: W [rows, K] times x [T, K]^T, both
// e4m3 codes with a power-of-two scale per 32 values, as the tensor cores take
// them (tcgen05 kind::mxf8f6f4 with a scale vector: exact products, scaled and
// summed in float32 in tensor memory).
//
// Features are the MMA's rows and tokens its columns (M = 128, N = kNT), so that
// one token costs a tile of 16 columns and not of 128 rows, and so that the 32
// values under one output scale are the 32 lanes of a warp.  A gated product's
// tile has 64 rows of its gate part and the same 64 of its up part, whose sums
// meet in shared memory.
//
// A CTA makes one output tile, over all of K or, where tiles are few, over one of
// the equal parts of K that a cluster's CTAs share; each then leaves its partial
// sums in its shared memory, and they sum up the results between them, in the
// order of the ranks.  With few tokens the product is bound by reading W: several
// CTAs an SM keep that read going while others start and end.
//
// Warp roles: 0 TMA of the codes (128-byte rows and swizzle), 1 MMA issuer, 2..5
// scales, 2..9 results.  The scales of a set of four steps (of 128 values of K) go
// by asynchronous copies into shared memory and from there into tensor memory,
// where each warp fills its quarter of the lanes: of a step's 8 columns the c-th
// holds the 4 bytes of W's row 32 c + lane, the (4 + c)-th those of that token.
// (With one set under way the loads' latency behind the codes' copies, microseconds,
// bound small products: one token through 8 experts of 12.6 MB 27.3 us, 24.9 with three.)
//
// Measured: 16 tokens x 4096 x 65536 (277 MB) 46.6 us, 6.0 TB/s with the launch, 64
// tokens 51.6; one token x 4096 x 4096 6.0 us, where an empty launch of this shape takes 0.8.
// Asking memory for W a window of steps ahead, row by row (bulk prefetches into
// L2), was slower: 31 to 45 us for 48 gated tokens x 4096 x 2 * 12288, 22.3 without.
#pragma once
#include <algorithm>
#include <atomic>
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
constexpr int kTileRows = 128; // rows of W per tile
constexpr int kResultWarps = 8;
constexpr int kMxThreads = (2 + kResultWarps) * 32;
constexpr int kMaxParts = 8;    // of K: CTAs of a (portable) cluster

// Set when a wait runs out in a kernel of the file that includes this.
__device__ int g_mx_timed_out;

// One thread that waits for what never comes, and so reports a wait that ran out.
__global__ void mx_wait_check_kernel() {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  abort_flag = 0;
  mbar_init(&bar, 1);
  mbar_fence_init();
  mbar_wait(&bar, 0, &abort_flag, &g_mx_timed_out, kDevWaitTimeout);
}
cudaError_t mx_wait_check(cudaStream_t stream) {
  mx_wait_check_kernel<<<1, 1, 0, stream>>>();
  return cudaGetLastError();
}

// (gelu has kernels of its own: chosen at run time beside the other activations, 128 tokens x 4096 x 4096 took 10.3 us with
// it, 9.3 so, and one token without it 6.2 instead of 6.0.)
enum MxMode { kLinear, kGelu, kGated, kMoeUp, kMoeDown };

// ---------------------------------------------------------------- instructions

// Instruction descriptor of kind::mxf8f6f4: e4m3 times e4m3, both K-major, scales
// as exponent bytes; sf: which of the 4 bytes of the scales' columns.
__host__ __device__ constexpr uint32_t idesc_sf(uint32_t sf) { return (sf << 4) | (sf << 29); }
__host__ __device__ constexpr uint32_t idesc_mx(uint32_t M, uint32_t N, uint32_t sf) {
  return ((N >> 3) << 17) | (1u << 23) | ((M >> 4) << 24) | idesc_sf(sf);
}
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// True in one thread of the (whole) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void prefetch_map(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Asynchronous copy of `bytes` (up to 4) bytes, zeros behind them.
__device__ __forceinline__ void cp_async4_zfill(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// An arrival that publishes nothing in memory.
__device__ __forceinline__ void mbar_arrive_relaxed(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// As if `bytes` bytes had arrived in the barrier's present phase.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
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
  bool give_up;            // for tests: every wait that is not over at once has run out
  int* status;             // of the call's workspace, or null: set when a wait runs out, as g_mx_timed_out
  MxEpilogue to;
  int64_t ld;              // features of an output row
  bool pairs;              // bf16 results and residual can be accessed two at a time
  bool publish;            // results are visible on the device before the CTAs end
  bool wide_scales;        // both sides' scale rows lie on 16-byte boundaries
  // mixture of experts
  const int32_t* ids;      // [T, topk]
  const float* weights;
  int topk, E;
  int slots;               // experts that a token tile can have at most
};

constexpr int kMaxMoeExperts = 512;
constexpr int kSetSteps = 4;  // steps whose scales go to tensor memory together
constexpr int kSets = 2;      // a ring of them

struct MxMisc {
  uint64_t full[6], empty[6], scaled[kSets], unscaled[kSets], done;
  uint32_t tmem;
  int abort_flag, active;
  uint32_t mask[kMaxMoeExperts / 32];
  uint16_t list[kMaxMoeExperts];
  float share[128];
  uint8_t routed[128];
};

template <int NT>
struct MxLay {
  static constexpr int kATile = kTileRows * kStepK;
  static constexpr int kStage = kATile + NT * kStepK;
  static constexpr int kCtas = 2;  // an SM
  static constexpr int kMisc = 1920;
  static constexpr int kRawSets = NT > 64 ? 3 : 4;  // sets of scales on their way
  static constexpr int kRaw = kRawSets * (kTileRows + NT) * 16;
  static constexpr int kFit = ((228 / kCtas - 1) * 1024 - 1024 - kMisc - kRaw) / kStage;
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kPartial = NT * kTileRows * 4;
  static constexpr int kOffRaw = kStages * kStage;
  static constexpr int kOffMisc = kOffRaw + kRaw;
  static constexpr int kSmem = kOffMisc + kMisc + 1024;
  static constexpr int kScaleCols = 8;          // of a step: W's block and the tokens'
  static constexpr int kNeed = NT + kSets * kSetSteps * kScaleCols;
  static constexpr int kCols = kNeed <= 128 ? 128 : 256;  // of tensor memory
  static_assert(kStages >= 2 && kStage % 1024 == 0 && kPartial <= kStages * kStage, "stages");
  static_assert(kNeed <= kCols && kCols * kCtas <= 512 && sizeof(MxMisc) <= kMisc, "limits");
};

// ---------------------------------------------------------------- the results' way out

__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.f + __expf(-x)); }

// x Phi(x), Phi the normal distribution, with the error of Phi's own value also where Phi is small (x (1 + erf(x / sqrt 2)) / 2
// is 4 % off at -5 in float32 and 0 below -5.6): with a = |x| and s = 1 / (1 + 0.26 a),
//   1 - Phi(a) = e^(-a^2 / 2) s P(s),
// as 1 / s times the rest is smooth from a = 0 to infinity.  P: least squares on 0 <= a <= 14, reweighted until the largest
// relative error, 2^-25, was least; in all within (x^2 + 6) 2^-23 of the value.  (2501 x 5120 x 13824 takes 120 us; by
// erfcf, whose branches the results' loop takes one after the other, 200, by 1 + erff 127.)
__device__ __forceinline__ float gelu(float x) {
  const float a = fabsf(x), s = __fdividef(1.f, fmaf(0.26f, a, 1.f));
  constexpr float kP[9] = {0.103759058f, 0.103016756f, 0.103030212f, 0.0510278568f, 0.160947397f,
                           -0.150948226f, 0.251490563f, -0.15282844f, 0.0305047967f};
  float r = kP[8];
#pragma unroll
  for (int k = 7; k >= 0; --k) r = fmaf(r, s, kP[k]);
  const float q = ex2_approx(a * a * -0.72134752f) * s * r;  // log2(e) / 2
  return x * (x < 0.f ? q : 1.f - q);
}

// Every activation but gelu.
__device__ __forceinline__ float activate(int kind, float x) {
  switch (kind) {
    case SMLA_ACT_RELU: return x < 0.f ? 0.f : x;  // (a NaN stays)
    case SMLA_ACT_SILU: return silu(x);
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

// Four tokens' results of a group of 32 features, one a lane, as codes: lane l gets
// those of token l % 4 and features l & ~3 .. l | 3, and that token's scale byte.
__device__ __forceinline__ uint32_t quantize4(float (&v)[4], uint32_t& scale) {
  const int lane = threadIdx.x & 31;
  uint32_t top[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) top[i] = __reduce_max_sync(kAllLanes, __float_as_uint(v[i]) & 0x7fffffffu);
  if (max(max(top[0], top[1]), max(top[2], top[3])) >= 0x7f800000u) {  // infinities and NaN are left out
#pragma unroll
    for (int i = 0; i < 4; ++i) top[i] = __reduce_max_sync(kAllLanes, mx_finite_bits(v[i]));
  }
  int e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e[i] = mx_exponent(top[i]);
    v[i] *= mx_pow2(-e[i]);
  }
  scale = (uint32_t)((lane & 2 ? (lane & 1 ? e[3] : e[2]) : (lane & 1 ? e[1] : e[0])) + 127);
  // bytes: this feature's 4 tokens; exchanged in fours of lanes for one token's 4 features
  uint32_t w = mx_e4m3x4(v[0], v[1], v[2], v[3]);
  uint32_t o = __shfl_xor_sync(kAllLanes, w, 1);
  w = __byte_perm(w, o, lane & 1 ? 0x3715 : 0x6240);
  o = __shfl_xor_sync(kAllLanes, w, 2);
  return __byte_perm(w, o, lane & 2 ? 0x3276 : 0x5410);
}
// Two tokens' results of this lane's feature as one token's of two features (lanes
// 2 k and 2 k + 1: features 2 k and 2 k + 1 of the first and of the second token).
__device__ __forceinline__ void pair_up(float first, float second, float& lo, float& hi) {
  const bool odd = threadIdx.x & 1;
  const float got = __shfl_xor_sync(kAllLanes, odd ? first : second, 1);
  lo = odd ? got : first;
  hi = odd ? second : got;
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
    uint32_t scale;
    const uint32_t w = quantize4(v, scale);
    const int i = lane & 3;
    if (i < n) {
      *reinterpret_cast<uint32_t*>(to.codes + (out_row + i) * p.ld + group + (lane & 28)) = w;
      if (lane < 4) to.scales[(out_row + i) * to.scale_stride + group / kMxGroup] = (uint8_t)scale;
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
      float lo, hi;
      pair_up(v[i], v[i + 1], lo, hi);
      const int k = i + (lane & 1);
      if (k >= n || even >= p.rows) continue;
      if (res) {
        // (a plain load: out may be the residual)
        const uint32_t r = *reinterpret_cast<const uint32_t*>(res + (out_row + k) * to.residual_stride + even);
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

// ---------------------------------------------------------------- the kernel

// grid: x = cluster rank + parts * row tile, y = token tile, z = expert slot (kMoeUp).
template <int MODE, int NT>
__global__ void __launch_bounds__(kMxThreads, MxLay<NT>::kCtas)
    mx_gemm_kernel(const __grid_constant__ MxParams p, const int parts, const __grid_constant__ CUtensorMap a_map,
                   const __grid_constant__ CUtensorMap b_map) {
  using L = MxLay<NT>;
  constexpr bool kGate = MODE == kGated || MODE == kMoeUp, kExperts = MODE == kMoeUp || MODE == kMoeDown;
  constexpr int kFeatures = kGate ? kTileRows / 2 : kTileRows;  // of a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  MxMisc& m = *reinterpret_cast<MxMisc*>(smem + L::kOffMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)blockIdx.x % parts, n0 = (int)blockIdx.x / parts * kFeatures;
  const int t0 = (int)blockIdx.y * NT, ntok = min(NT, p.T - t0);
  volatile int* abort_flag = &m.abort_flag;

  if (tid == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&m.full[s], 1);
      mbar_init(&m.empty[s], 1);
    }
    for (int s = 0; s < kSets; ++s) {
      mbar_init(&m.scaled[s], 4);
      mbar_init(&m.unscaled[s], 1);
    }
    mbar_init(&m.done, 1);
    m.abort_flag = p.give_up;
    mbar_fence_init();
  }
  if (tid == 96) {
    prefetch_map(&a_map);
    prefetch_map(&b_map);
  }
  if (warp == 1) {
    tmem_alloc(&m.tmem, L::kCols);
    tmem_relinquish();
  }
  if (kExperts && tid < kMaxMoeExperts / 32) m.mask[tid] = 0u;
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
  int total = steps, expert = 0;
  if (kExperts) {
    // the experts that this tile's tokens go to, in order
    for (int i = tid; i < ntok * p.topk; i += kMxThreads) {
      const int id = __ldg(p.ids + (int64_t)t0 * p.topk + i);
      if (id >= 0 && id < p.E) atomicOr(&m.mask[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
    for (int e = tid; e < kMaxMoeExperts; e += kMxThreads) {
      int before = 0, all = 0;  // experts taken of the words before e's, and of all
#pragma unroll
      for (int w = 0; w < kMaxMoeExperts / 32; ++w) {
        const int count = __popc(m.mask[w]);
        before += w < e / 32 ? count : 0;
        all += count;
      }
      const uint32_t word = m.mask[e / 32], bit = 1u << (e % 32);
      if (word & bit) m.list[before + __popc(word & (bit - 1u))] = (uint16_t)e;
      if (e == 0) m.active = all;
    }
    __syncthreads();
    if (MODE == kMoeUp) {
      const bool idle = (int)blockIdx.z >= m.active;  // the same for a whole cluster
      expert = idle ? 0 : m.list[blockIdx.z];
      if (idle) total = 0;
    } else {
      total = m.active * steps;
    }
  }
  // Parts of whole sets where the scales of a set can be copied at once: 16 bytes of a row, on 16-byte boundaries.
  const bool wide = p.wide_scales && (MODE != kMoeDown || steps % kSetSteps == 0);
  const int unit = wide ? kSetSteps : 1;
  const int units = (total + unit - 1) / unit;
  const int k0 = (int)((int64_t)units * rank / parts) * unit;
  const int n = min(total, (int)((int64_t)units * (rank + 1) / parts) * unit) - k0;
  const int slot0 = MODE == kMoeUp ? (int)(blockIdx.y * p.slots + blockIdx.z) : (int)blockIdx.y * p.slots;
  // Step it's place in its row, and its expert's place in the list.
  auto in_row = [&](int it) { return MODE == kMoeDown ? it % steps : it; };
  auto in_list = [&](int it) { return MODE == kMoeDown ? it / steps : 0; };
  auto expert_of = [&](int it) { return MODE == kMoeDown ? (int)m.list[it / steps] : expert; };

#define MX_WAIT(bar, parity) mbar_wait(&(bar), (parity), abort_flag, &g_mx_timed_out, kDevWaitTimeout)
  bool dead = false;
  int issued = 0;  // copies of codes (warp 0)
  if (warp == 0) {
    // ---------------------------------------------------------------- codes
    auto load_a = [&](int i, int s) {
      const int it = k0 + i, x = in_row(it) * kStepK, y = expert_of(it) * (kGate ? 2 : 1) * p.rows + n0;
      const uint32_t stage = smem_u32(smem + s * L::kStage);
      mbar_arrive_expect_tx(&m.full[s], (uint32_t)L::kStage);
      tma_load_2d(stage, &a_map, x, y, &m.full[s]);
      if (kGate) tma_load_2d(stage + L::kATile / 2, &a_map, x, y + p.rows, &m.full[s]);
    };
    auto load_b = [&](int i, int s) {
      const int it = k0 + i;
      tma_load_2d(smem_u32(smem + s * L::kStage) + L::kATile, &b_map, in_row(it) * kStepK,
                  MODE == kMoeDown ? (slot0 + in_list(it)) * NT : t0, &m.full[s]);
    };
    const int early = MODE == kMoeDown ? min(n, L::kStages) : 0;
    if (MODE == kMoeDown) {
      if (lane == 0)
        for (int i = 0; i < early; ++i) load_a(i, i);
      __syncwarp();
      grid_dependency_wait();
      if (lane == 0)
        for (int i = 0; i < early; ++i) load_b(i, i);
    }
    int s = early % L::kStages;
    issued = early;
    uint32_t phase = early == L::kStages ? 1u : 0u;  // of the fillings of stage s
    bool ok = true;
    for (int i = early; i < n && ok; ++i) {
      if (i >= L::kStages) ok = MX_WAIT(m.empty[s], phase ^ 1u);
      ok = __all_sync(kAllLanes, ok);
      if (!ok) break;
      if (lane == 0) {
        load_a(i, s);
        load_b(i, s);
      }
      __syncwarp();
      ++issued;
      if (++s == L::kStages) s = 0, phase ^= 1u;
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    // The whole warp goes through the loop and elects the issuing thread, so that operands lie in uniform registers.
    constexpr uint32_t kHi = sdesc_hi(1024, kLayoutSw128);
    const uint32_t lo0 = sdesc_lo(smem_u32(smem), 16);
    int s = 0, set = 0;
    uint32_t phase = 0, set_phase = 0;
    bool ok = true;
    for (int i0 = 0; i0 < n && ok; i0 += kSetSteps) {
      if (!(ok = MX_WAIT(m.scaled[set], set_phase))) break;
      const int left = min(kSetSteps, n - i0);
      uint32_t sf = tmem + NT + set * kSetSteps * L::kScaleCols;
      for (int k = 0; k < left; ++k, sf += L::kScaleCols) {
        if (!(ok = MX_WAIT(m.full[s], phase))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t lo = lo0 + (uint32_t)s * (L::kStage >> 4);
#pragma unroll
          for (int kk = 0; kk < kStepK / 32; ++kk)
            mma_mx(tmem, sdesc_join<kHi>(lo + 2 * kk), sdesc_join<kHi>(lo + (L::kATile >> 4) + 2 * kk),
                   idesc_mx(kTileRows, NT, kk), sf, sf + 4, kk > 0 ? 1u : (uint32_t)((i0 | k) != 0));
          mma_commit(&m.empty[s]);
          if (k + 1 == left) mma_commit(&m.unscaled[set]);
        }
        __syncwarp();
        if (++s == L::kStages) s = 0, phase ^= 1u;
      }
      if (++set == kSets) set = 0, set_phase ^= 1u;
    }
    if (elect_one()) mma_commit(&m.done);
    __syncwarp();
    mbar_wait_drain(&m.done, 0);
  } else if (warp < 6) {
    // ---------------------------------------------------------------- scales
    // Thread r copies row r of W's 128 and, below NT, of the tokens', a set's 16 bytes, into a ring of kRawSets, all but
    // one of them under way: behind the codes' copies a load takes microseconds.
    const int q = warp & 3, r = 32 * q + lane;
    const int groups = p.K / kMxGroup;
    constexpr int kRaw = (kTileRows + NT) * 16, kRawSets = L::kRawSets;
    const uint32_t raw = smem_u32(smem + L::kOffRaw);
    const int f = n0 + (kGate ? r % kFeatures : r);
    const int64_t a_row = (kGate && r >= kFeatures ? p.rows : 0) + f, per_expert = (int64_t)(kGate ? 2 : 1) * p.rows;
    auto copy = [&](uint32_t dst, const uint8_t* row, int x, bool there) {  // from step x of a row on; behind its end zeros
      const int left = there ? groups - 4 * x : 0;
      if (wide) cp_async16_zfill(dst, there ? row + 4 * x : p.a_scale, (uint32_t)min(max(left, 0), 16));
      else cp_async4_zfill(dst, there ? row + 4 * x : p.a_scale, (uint32_t)min(max(left, 0), 4));
    };
    auto copy_a = [&](int i0, int slot) {
      for (int k = 0; k < kSetSteps && i0 + k < n; k += wide ? kSetSteps : 1) {
        const int it = k0 + i0 + k;
        copy(raw + slot * kRaw + 16 * r + 4 * k, p.a_scale + (expert_of(it) * per_expert + a_row) * p.a_scale_stride, in_row(it),
             f < p.rows);
      }
    };
    auto copy_b = [&](int i0, int slot) {
      if (r >= NT) return;
      for (int k = 0; k < kSetSteps && i0 + k < n; k += wide ? kSetSteps : 1) {
        const int it = k0 + i0 + k;
        const int64_t row = MODE == kMoeDown ? (int64_t)(slot0 + in_list(it)) * NT + r : t0 + r;
        copy(raw + slot * kRaw + 16 * (kTileRows + r) + 4 * k, p.b_scale + row * p.b_scale_stride, in_row(it), r < ntok);
      }
    };
#pragma unroll
    for (int j = 0; j < kRawSets - 1; ++j) copy_a(j * kSetSteps, j);
    if (MODE == kMoeDown) grid_dependency_wait();
#pragma unroll
    for (int j = 0; j < kRawSets - 1; ++j) {
      copy_b(j * kSetSteps, j);
      cp_async_commit();  // (the first one's group has all of W's scales)
    }
    if (MODE == kMoeUp && r < NT) {
      // the weight that this thread's token gives the expert, while the first copies are under way
      float w = 0.f;
      bool any = false;
      const int64_t first = (int64_t)(t0 + r) * p.topk;
#pragma unroll 8
      for (int k = 0; k < (r < ntok ? p.topk : 0); ++k) {
        const int id = __ldg(p.ids + first + k);
        const float x = __ldg(p.weights + first + k);
        if (id == expert) w += x, any = true;
      }
      m.share[r] = w;
      m.routed[r] = any;
    }
    const uint32_t to = tmem + ((uint32_t)(32 * q) << 16) + NT;
    int set = 0, slot = 0;
    uint32_t phase = 0;
    for (int i0 = 0; i0 < n; i0 += kSetSteps) {
      cp_async_wait<kRawSets - 2>();
      named_bar_sync(1, 128);  // everyone's copies of this set are there, and everyone has read the one before
      const int before = slot == 0 ? kRawSets - 1 : slot - 1;
      copy_a(i0 + (kRawSets - 1) * kSetSteps, before);
      copy_b(i0 + (kRawSets - 1) * kSetSteps, before);
      cp_async_commit();
      if (!dead && i0 >= kSets * kSetSteps) dead = __any_sync(kAllLanes, !MX_WAIT(m.unscaled[set], phase ^ 1u));
      tc_fence_after();
      // lane l: four steps' words of rows l, l + 32, .. of W's block and of the tokens'
      constexpr int kB = NT / 32 > 0 ? NT / 32 : 1;
      uint4 w[4], x[4] = {};
#pragma unroll
      for (int c = 0; c < 4; ++c) w[c] = ld_shared_v4(raw + slot * kRaw + 16 * (32 * c + lane));
#pragma unroll
      for (int c = 0; c < kB; ++c) x[c] = ld_shared_v4(raw + slot * kRaw + 16 * (kTileRows + (NT < 32 ? lane % NT : 32 * c + lane)));
      if (!dead) {
        const uint32_t at = to + set * kSetSteps * L::kScaleCols;
        const uint32_t first[16] = {w[0].x, w[1].x, w[2].x, w[3].x, x[0].x, x[1].x, x[2].x, x[3].x,
                                    w[0].y, w[1].y, w[2].y, w[3].y, x[0].y, x[1].y, x[2].y, x[3].y};
        const uint32_t second[16] = {w[0].z, w[1].z, w[2].z, w[3].z, x[0].z, x[1].z, x[2].z, x[3].z,
                                     w[0].w, w[1].w, w[2].w, w[3].w, x[0].w, x[1].w, x[2].w, x[3].w};
        tmem_st16(at, first);
        tmem_st16(at + 16, second);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(&m.scaled[set]);
      }
      if (++set == kSets) set = 0, phase ^= 1u;
      if (++slot == kRawSets) slot = 0;
    }
    cp_async_wait<0>();  // none may land later, in what is then something else
  }
  if (warp >= 2) {
    dead = __any_sync(kAllLanes, dead || !MX_WAIT(m.done, 0));
    tc_fence_after();
  }
#undef MX_WAIT

  // ---------------------------------------------------------------- results
  const int q = warp & 3, half = (warp - 2) >> 2;  // two warps have the same lanes of tensor memory
  const MxOut kind = MODE == kMoeUp ? kOutCodes : out_kind(p);
  // Tokens c .. c + 3 of the group of 32 features `group` (of the tile), one a lane; biases b0, b1.
  auto finish = [&](auto out, const float (&v)[4], const float (&up)[4], float b0, float b1, int group, int c) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = v[i] + b0;
      if (kGate) y[i] = silu(y[i]) * (up[i] + b1);
      else if (MODE == kGelu) y[i] = gelu(y[i]);
      if (MODE == kMoeUp) y[i] = m.routed[c + i] ? y[i] * m.share[c + i] : 0.f;  // (tokens behind the last are not routed)
    }
    if (MODE == kLinear && p.to.activation != SMLA_ACT_NONE)
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = activate(p.to.activation, y[i]);
    const int64_t row = MODE == kMoeUp ? (int64_t)slot0 * NT + c : t0 + c;
    write_out<decltype(out)::value>(p, y, n0 + 32 * group + lane, n0 + 32 * group, row, ntok - c);
  };
  auto biases = [&](int group, float& b0, float& b1) {
    const int f = n0 + 32 * group + lane;
    const bool biased = !kExperts && p.to.bias != nullptr && f < p.rows;
    b0 = biased ? bias_at(p.to, f) : 0.f;
    b1 = kGate && biased ? bias_at(p.to, (int64_t)p.rows + f) : 0.f;
  };
  // body(out) for the way that results go
  auto by_kind = [&](auto body) {
    if (kind == kOutCodes) body(std::integral_constant<MxOut, kOutCodes>{});
    else if (kind == kOutPairs) body(std::integral_constant<MxOut, kOutPairs>{});
    else body(std::integral_constant<MxOut, kOutSingle>{});
  };
  // 16 columns of this warp's lanes
  auto columns = [&](int c, uint32_t (&w)[16]) {
    tmem_ld16(tmem + ((uint32_t)(32 * q) << 16) + c, w);
    tmem_ld_wait();
    reg_fence16(w);
    if (n == 0)  // no part of K: nothing has been summed
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = 0u;
  };
  if (MODE == kMoeUp && total == 0) {
    // no such expert: nothing to compute, nothing to write
  } else if (parts == 1 && !kGate) {
    if (warp >= 2 && !dead) {
      float b0, b1;
      biases(q, b0, b1);
      by_kind([&](auto out) {
#pragma unroll 1
        for (int c = 16 * half; c < ntok; c += 32) {
          uint32_t w[16];
          columns(c, w);
#pragma unroll
          for (int h = 0; h < 16; h += 4) {
            const float v[4] = {__uint_as_float(w[h]), __uint_as_float(w[h + 1]), __uint_as_float(w[h + 2]),
                                __uint_as_float(w[h + 3])};
            if (c + h < ntok) finish(out, v, v, b0, b1, q, c + h);
          }
        }
      });
    }
  } else {
    float* part = reinterpret_cast<float*>(smem);  // [column][row]; every copy and MMA has ended
    if (warp >= 2 && !dead) {
#pragma unroll 1
      for (int c = 16 * half; c < ntok; c += 32) {
        uint32_t w[16];
        columns(c, w);
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * kTileRows + 32 * q + lane] = __uint_as_float(w[i]);
      }
    }
    __syncwarp();
    if (parts > 1) cluster_sync_all();
    else __syncthreads();
    if (warp >= 2 && !dead) {
      // Blocks of kBlock tokens by 32 features, dealt to the cluster's warps.  (Blocks of 16, with more chains of
      // operations at once, are more code that each CTA runs once, and took longer: 4.9 us against 3.9 for 48 tokens.)
      constexpr int kGroups = kFeatures / 32, kBlock = 4;
      const int blocks = (ntok + kBlock - 1) / kBlock * kGroups;
      by_kind([&](auto out) {
#pragma unroll 1
        for (int u = (warp - 2) * parts + rank; u < blocks; u += kResultWarps * parts) {
          const int group = u % kGroups, c0 = u / kGroups * kBlock;
          float b0, b1;
          biases(group, b0, b1);
          float v[kBlock], up[kBlock];
          auto sum = [&](float (&to)[kBlock], uint32_t at) {
#pragma unroll
            for (int i = 0; i < kBlock; ++i) to[i] = 0.f;
            for (int o = 0; o < parts; o += 4) {
              float x[4][kBlock];
#pragma unroll
              for (int k = 0; k < 4; ++k)  // all loads before the first sum
                if (o + k < parts) {
                  const uint32_t from = parts > 1 ? mapa_shared(at, (uint32_t)(o + k)) : at;
#pragma unroll
                  for (int i = 0; i < kBlock; ++i) x[k][i] = ld_cluster_f32(from + 4 * kTileRows * i);
                }
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (o + k < parts)
#pragma unroll
                  for (int i = 0; i < kBlock; ++i) to[i] += x[k][i];
            }
          };
          const uint32_t mine = smem_u32(part) + 4 * (c0 * kTileRows + 32 * group + lane);
          sum(v, mine);
          if (kGate) sum(up, mine + 4 * kFeatures);
#pragma unroll
          for (int h = 0; h < kBlock; h += 4) {
            const float a[4] = {v[h], v[h + 1], v[h + 2], v[h + 3]};
            const float g[4] = {kGate ? up[h] : 0.f, kGate ? up[h + 1] : 0.f, kGate ? up[h + 2] : 0.f, kGate ? up[h + 3] : 0.f};
            if (c0 + h < ntok) finish(out, a, g, b0, b1, group, c0 + h);
          }
        }
      });
    }
    __syncwarp();
    if (parts > 1) cluster_sync_relaxed();  // no CTA leaves while another reads its sums
  }
  if (!kExperts && p.publish && warp >= 2) __threadfence();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
  if (*abort_flag) {
    // A wait ran out, and what it was for may still be under way: no copy may land once this CTA's shared memory is
    // another's.  (The MMAs have been waited for, and the scales' copies.)
    if (warp == 0)
      for (int i = max(0, issued - L::kStages); i < issued; ++i)
        mbar_wait_drain(&m.full[i % L::kStages], (i / L::kStages) & 1);
    if (tid == 0) {
      atomicExch(&g_mx_timed_out, kDevWaitTimeout);
      if (p.status) atomicExch(p.status, kDevWaitTimeout);  // (whatever an uninitialised workspace held)
    }
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
bool rows16(const uint8_t* p, int64_t stride) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 16 == 0; }

// Codes [rows, K] in boxes of 128 bytes of box_rows rows.
cudaError_t code_map(CUtensorMap* map, const void* base, int64_t rows, int64_t K, int64_t stride, int box_rows) {
  return byte_map(map, base, rows, K, stride, kStepK, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// The kernel's shared memory, once per device (a fifth of a microsecond, where a small call takes five); `done`: which.
template <typename F>
cudaError_t allow_smem(F* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (e != cudaSuccess || (done.load(std::memory_order_relaxed) & bit)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <int MODE, int NT>
cudaError_t launch_mx(const MxParams& p, int parts, int64_t row_tiles, int64_t token_tiles, int slots,
                      const CUtensorMap& a_map, const CUtensorMap& b_map, cudaStream_t stream) {
  if (row_tiles * parts > INT32_MAX || token_tiles > 65535 || slots > 65535) return cudaErrorInvalidValue;
  auto kernel = mx_gemm_kernel<MODE, NT>;
  constexpr int smem = MxLay<NT>::kSmem;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(kernel, smem, allowed);
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

// Parts of K, a power of two: as many as leave each 8 steps, up to two CTAs an SM, and then 4 steps, up to one.  One token,
// 4 parts | 8: N x K = 4096 x 4096 5.8 | 6.7 us, 2048 x 2048 4.9 | 6.2, 4096 x 12288 10.7 | 9.8, 1536 x 7168 7.8 | 6.4;
// 8192 x 4096 2 parts 8.1, 4 parts 7.4.
int split_k(int64_t tiles, int64_t steps, int num_sms) {
  int parts = 1;
  while (parts < kMaxParts) {
    const int64_t ctas = 2 * parts * tiles, left = steps / (2 * parts);
    if (!((left >= 8 && ctas <= 2 * (int64_t)num_sms) || (left >= 4 && ctas <= num_sms))) break;
    parts *= 2;
  }
  return parts;
}

}  // namespace

}  // namespace smla
