// The experts of each token from its router logits: scores by softmax or
// sigmoid, a selection bias, groups of experts of which the best are kept, the
// topk largest, and their weights.
//
// One warp per token; what it ranks by lies in registers, expert 32 i + l in
// lane l, and a round of the selection is a maximum over the warp of ordered
// bits, then the lowest index that has it.  Without bias and groups the logits
// themselves are ranked, so float32 decides exactly.  With them what is ranked is
// computed, and near ties could fall either way: where two neighbours of the
// ranking, as far as it decides, are nearer than the computation's error, those
// taken (and those that follow as closely) are ordered by scores of 64 bits, one a
// lane; near ties of groups and of softmax scores rank the token again in 64 bits.
// (All scores in 64 bits would take an exponential of 64 bits per expert, at a
// sixtieth of the rate: 48 tokens with one near tie took 19 us so.)  The call is
// bound by the launch and the chain of rounds: 48 tokens x 256 experts in 8 groups
// 7 us (10 with near ties), 9000 x 64 5 to 6.5 us, 9000 x 256 in groups 25 us.
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sm103_ptx.cuh"
#include "smla_kernels.h"

namespace smla {

namespace {

constexpr uint32_t kLanes = 0xffffffffu;
constexpr int kRouteWarps = 4;

// Bits ordered as the values are, above 0; 0 for NaN and -infinity, which are
// never taken, and for what has been taken.
__device__ __forceinline__ uint32_t order_bits(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);  // (-0 is 0)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_bits(double x) {
  if (!(x > -INFINITY)) return 0u;
  const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
  return b >> 63 ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ float value_of(uint32_t b) { return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b); }
__device__ __forceinline__ double value_of(uint64_t b) {
  return __longlong_as_double((long long)(b >> 63 ? b & ~(1ull << 63) : ~b));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kLanes, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(kLanes, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(kLanes, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ float score_of(bool sigmoid, float x, float top, float inv_sum) {
  return sigmoid ? 1.f / (1.f + expf(-x)) : expf(x - top) * inv_sum;
}

// How far a float32 score plus bias may be from the exact one, in units of 2^-24 of
// the score (at most 1): 2 for the exponential, 1 for the quotient and one of the
// sum with the bias; by sigmoid 1 more for the sum with 1 (6 in all, 8 are taken), by
// softmax 1 for the argument's rounding (s |x - top| < 1/2) and up to 21 for the sum
// of 512 exponentials (32 are taken).
__device__ __forceinline__ float slack(bool sigmoid, float x) { return (sigmoid ? 0x1p-21f : 0x1p-19f) * (1.f + fabsf(x)); }

// Below this, in logits from 0 or from the largest, float32 may hold a score with fewer bits than normal numbers have:
// e^-87.3 is the smallest of these, and a sum of 512 divides by up to e^6.3.
constexpr float kSmallScore = -80.f;

struct Taken {
  int id;            // lane k: the k-th expert, -1: there was none
  int count;         // how many there are: topk, and those that follow by less than their error
  bool near;         // two neighbours of them are nearer than that
  bool groups_near;  // as are the last group kept and the first left
};

// Ranks a token's experts (keys[i]: of expert 32 i + lane) and takes topk of
// them, and with `check` also those that follow too closely.  `scratch`: E keys of
// shared memory, used with groups.
template <int R, typename Bits>
__device__ __forceinline__ Taken take(const MoeRouteArgs& a, Bits (&keys)[R], Bits* scratch, bool check) {
  const int lane = threadIdx.x & 31;
  Taken got{-1, 0, false, false};
  if (a.groups > 1) {
    const int size = a.E / a.groups;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (32 * i + lane < a.E) scratch[32 * i + lane] = keys[i];
    __syncwarp();
    // each group's two largest, by as many lanes as there are for it (a power of two); their sum's key
    const int share = 32 - __clz(32 / a.groups) - 1, lanes = 1 << share, mine = lane >> share;
    Bits first = 0, second = 0;
    if (mine < a.groups)
      for (int i = lane & (lanes - 1); i < size; i += lanes) {
        const Bits k = scratch[mine * size + i];
        second = k > first ? first : k > second ? k : second;
        first = k > first ? k : first;
      }
    for (int d = 1; d < lanes; d *= 2) {
      const Bits f = __shfl_xor_sync(kLanes, first, d), g = __shfl_xor_sync(kLanes, second, d);
      const Bits less = f < first ? f : first, other = g > second ? g : second;
      first = f > first ? f : first;
      second = less > other ? less : other;
    }
    Bits group = second ? order_bits(value_of(first) + value_of(second)) : 0;
    // The error of a group's sum is its two addends', which may be far larger than it; the largest of all groups' counts.
    float error = check && second ? slack(a.sigmoid, (float)value_of(first)) + slack(a.sigmoid, (float)value_of(second)) : 0.f;
    if (check) error = __uint_as_float(__reduce_max_sync(kLanes, __float_as_uint(error)));
    __syncwarp();
    uint32_t kept = 0u;
    Bits last = 0;
    for (int r = 0; r <= a.topk_groups; ++r) {  // one more, to see how near it is
      const Bits top = warp_max(group);
      if (check && r == a.topk_groups && top) {
        got.groups_near = (float)value_of(last) - (float)value_of(top) <= 2.f * error;
      }
      if (r == a.topk_groups || !top) break;
      const int g = (__ffs(__ballot_sync(kLanes, group == top)) - 1) >> share;
      kept |= 1u << g;
      if (mine == g) group = 0;
      last = top;
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (32 * i + lane < a.E && !(kept >> ((32 * i + lane) / size) & 1u)) keys[i] = 0;
  }
  Bits last = 0;
  for (int r = 0; r < 32; ++r) {
    if (r >= a.topk && !check) break;
    Bits best = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) best = keys[i] > best ? keys[i] : best;
    const Bits top = warp_max(best);
    if (!top) break;
    if (check && r > 0) {
      const float lo = (float)value_of(top), hi = (float)value_of(last);
      const bool near = hi - lo <= slack(a.sigmoid, lo) + slack(a.sigmoid, hi);
      if (r >= a.topk && !near) break;
      got.near |= near;
    }
    uint32_t at = 0xffffffffu;
#pragma unroll
    for (int i = R - 1; i >= 0; --i)
      if (keys[i] == top) at = (uint32_t)(32 * i + lane);
    const int e = (int)__reduce_min_sync(kLanes, at);
    if (lane == r) got.id = e;
    got.count = r + 1;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (32 * i + lane == e) keys[i] = 0;
    last = top;
  }
  if (check && got.count == 32) {  // whether one more follows as closely
    Bits best = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) best = keys[i] > best ? keys[i] : best;
    const Bits top = warp_max(best);
    const float lo = top ? (float)value_of(top) : 0.f, hi = (float)value_of(last);
    got.near |= top && hi - lo <= slack(a.sigmoid, lo) + slack(a.sigmoid, hi);
  }
  return got;
}

// The order of the taken ones in 64 bits, by sigmoid: each lane its own expert's score, and its place among the others.
template <typename X>
__device__ __noinline__ int order_64(const MoeRouteArgs& a, const X* logits, int id, uint64_t* scratch) {
  const int lane = threadIdx.x & 31;
  uint64_t key = 0;
  if (id >= 0) key = order_bits(1. / (1. + exp(-(double)(float)logits[id])) + (a.bias ? (double)a.bias[id] : 0.));
  int place = 0;
  for (int i = 0; i < 32; ++i) {
    const uint64_t k = __shfl_sync(kLanes, key, i);
    const int other = __shfl_sync(kLanes, id, i);
    place += k > key || (k == key && other >= 0 && other < id);
  }
  __syncwarp();
  int* ids = reinterpret_cast<int*>(scratch);
  ids[lane] = -1;
  __syncwarp();
  if (id >= 0) ids[place] = id;
  __syncwarp();
  return ids[lane];
}

// The same in 64 bits, from the logits on.
template <int R, typename X>
__device__ __noinline__ int take_64(const MoeRouteArgs& a, const X* logits, uint64_t* scratch) {
  const int lane = threadIdx.x & 31;
  uint64_t keys[R];
  double x[R], top = -INFINITY, sum = 0.;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    x[i] = 32 * i + lane < a.E ? (double)(float)logits[32 * i + lane] : -INFINITY;
    if (x[i] > top) top = x[i];
  }
  if (!a.sigmoid) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmax(top, __shfl_xor_sync(kLanes, top, d));
#pragma unroll
    for (int i = 0; i < R; ++i) sum += x[i] > -INFINITY ? exp(x[i] - top) : 0.;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kLanes, sum, d);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = 32 * i + lane;
    keys[i] = 0;
    if (e < a.E && x[i] > -INFINITY)
      keys[i] = order_bits((a.sigmoid ? 1. / (1. + exp(-x[i])) : exp(x[i] - top) / sum) + (a.bias ? (double)a.bias[e] : 0.));
  }
  return take<R, uint64_t>(a, keys, scratch, false).id;
}

template <int R, typename X>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const __grid_constant__ MoeRouteArgs a) {
  __shared__ uint64_t scratch[kRouteWarps][32 * R];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  grid_dependency_wait();
  if (t >= a.T) return;
  const X* logits = static_cast<const X*>(a.logits) + t * a.E;
  float x[R], top = -INFINITY;
#pragma unroll
  for (int i = 0; i < R; ++i) x[i] = 32 * i + lane < a.E ? (float)logits[32 * i + lane] : -INFINITY;
#pragma unroll
  for (int i = 0; i < R; ++i) top = fmaxf(top, x[i]);
  const bool computed = a.bias != nullptr || a.groups > 1;  // what is ranked
  float sum = 0.f, inv = 1.f;
  if (!a.sigmoid) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kLanes, top, d));
    if (computed || !a.renormalize) {
#pragma unroll
      for (int i = 0; i < R; ++i) sum += x[i] > -INFINITY ? expf(x[i] - top) : 0.f;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kLanes, sum, d);
      inv = 1.f / sum;
    }
  }
  uint32_t keys[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = 32 * i + lane;
    float rank = x[i];
    if (computed && x[i] > -INFINITY) rank = score_of(a.sigmoid, x[i], top, inv) + (a.bias && e < a.E ? __ldg(a.bias + e) : 0.f);
    keys[i] = e < a.E && x[i] > -INFINITY ? order_bits(rank) : 0u;
  }
  const Taken got = take<R, uint32_t>(a, keys, reinterpret_cast<uint32_t*>(scratch[warp]), computed);
  int id = got.id;
  if (got.groups_near || (got.near && (!a.sigmoid || got.count == 32))) {
    __syncwarp();
    id = take_64<R, X>(a, logits, scratch[warp]);
  } else if (got.near) {
    id = order_64<X>(a, logits, id, scratch[warp]);
  }
  if (lane >= a.topk) id = -1;
  // lane k: the k-th expert's weight
  const float logit = id >= 0 ? (float)logits[id] : -INFINITY;
  float w = id >= 0 ? score_of(a.sigmoid, logit, top, inv) : 0.f;
  if (a.renormalize) {
    if (__any_sync(kLanes, id >= 0 && (a.sigmoid ? logit : logit - top) < kSmallScore)) {
      // Shares are ratios, whatever the scores' size: all times what makes the largest taken one about 1.
      float most = logit;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(kLanes, most, d));
      if (a.sigmoid) most = fminf(most, 0.f);
      w = 0.f;
      if (id >= 0) w = !a.sigmoid ? expf(logit - most) : logit < 0.f ? expf(logit - most) / (1.f + expf(logit)) : 1.f / (1.f + expf(-logit));
    }
    float all = w;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(kLanes, all, d);
    w = all > 0.f ? w / all : id >= 0 ? w : 0.f;
  }
  if (lane < a.topk) {
    a.ids[t * a.topk + lane] = id;
    a.weights[t * a.topk + lane] = id >= 0 ? w * a.scale : 0.f;
  }
}

template <int R, typename X>
cudaError_t launch_route(const MoeRouteArgs& a, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(((int64_t)a.T + kRouteWarps - 1) / kRouteWarps));
  cfg.blockDim = dim3(32 * kRouteWarps);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, route_kernel<R, X>, a);
}

template <typename X>
cudaError_t launch_experts(const MoeRouteArgs& a, cudaStream_t stream) {
  if (a.E <= 64) return launch_route<2, X>(a, stream);
  if (a.E <= 128) return launch_route<4, X>(a, stream);
  if (a.E <= 256) return launch_route<8, X>(a, stream);
  return launch_route<16, X>(a, stream);
}

}  // namespace

cudaError_t launch_moe_route(const MoeRouteArgs& a, cudaStream_t stream) {
  return a.logits_f32 ? launch_experts<float>(a, stream) : launch_experts<__nv_bfloat16>(a, stream);
}

}  // namespace smla
