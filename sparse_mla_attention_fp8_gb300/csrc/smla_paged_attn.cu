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
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "sm103_ptx.cuh"
#include "smla_common.cuh"
#include "smla_kernels.h"
#include "smla_paged.cuh"

namespace smla {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float e4m3(uint8_t c) {
  __nv_fp8_e4m3 x;
  x.__x = c;
  return (float)x;
}

// One CTA per (token, K/V head): the keys' blocks in turn through shared
// memory as floats, an online softmax per head.
template <int D>
__global__ void __launch_bounds__(kThreads) paged_attn_simple_kernel(const __grid_constant__ PagedAttnArgs a) {
  extern __shared__ float sm[];
  const int G = a.H / a.HK, t = (int)blockIdx.x, g = (int)blockIdx.y, tid = threadIdx.x;
  float* qs = sm;                // [G][D]
  float* acc = qs + G * D;       // [G][D]
  float* kv = acc + G * D;       // [64][D + 1]
  float* p = kv + kBlock * (D + 1);  // [G][64]
  float* m = p + G * kBlock;     // [G]
  float* l = m + G;              // [G]
  float* alpha = l + G;          // [G]
  const int r = search_units(a.R, t, [&](int i) { return clamp_start(a.query_start, i, a.T); });
  const int t0 = clamp_start(a.query_start, r, a.T), t1 = clamp_start(a.query_start, r + 1, a.T);
  if (t < t0 || t >= t1) return;
  const int64_t len = a.seq_lens[r], pos = len - t1 + t;
  int64_t hi = pos + 1, lo = 0;
  if (a.prefix_lens) hi = max(hi, (int64_t)a.prefix_lens[r]);
  hi = min(hi, min(len, (int64_t)a.MB * kBlock));
  if (a.window > 0) lo = max(lo, pos - a.window + 1);
  if (a.doc_start) lo = max(lo, (int64_t)a.doc_start[t]);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + t * a.q_stride + (int64_t)g * G * D;
  for (int i = tid; i < G * D; i += kThreads) {
    qs[i] = __bfloat162float(q[i]);
    acc[i] = 0.f;
  }
  for (int i = tid; i < G; i += kThreads) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
  __syncthreads();
  for (int64_t j = lo / kBlock; j * kBlock < hi; ++j) {
    const int b = a.block_table[(int64_t)r * a.MB + j];
    if (b < 0 || b >= a.NB) continue;
    const int64_t bh = (int64_t)b * a.HK + g;
    const uint8_t* kp = a.k_cache + bh * kBlock * D;
    for (int i = tid; i < kBlock * D; i += kThreads) kv[i / D * (D + 1) + i % D] = e4m3(kp[i]);
    __syncthreads();
    const float ks = a.k_scale[bh];
    for (int i = tid; i < G * kBlock; i += kThreads) {
      const int h = i / kBlock, key = i % kBlock;
      const int64_t kpos = j * kBlock + key;
      float x = -INFINITY;
      if (kpos >= lo && kpos < hi) {
        x = 0.f;
        for (int d = 0; d < D; ++d) x = fmaf(qs[h * D + d], kv[key * (D + 1) + d], x);
        x *= a.sm_scale * ks;
        if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
        if (a.alibi_slopes) x -= a.alibi_slopes[g * G + h] * (float)llabs(pos - kpos);
      }
      p[i] = x;
    }
    __syncthreads();
    for (int h = tid; h < G; h += kThreads) {
      float mx = m[h];
      for (int k = 0; k < kBlock; ++k) mx = fmaxf(mx, p[h * kBlock + k]);
      const float base = mx == -INFINITY ? 0.f : mx;
      float s = 0.f;
      for (int k = 0; k < kBlock; ++k) s += p[h * kBlock + k] = expf(p[h * kBlock + k] - base);
      alpha[h] = expf(m[h] - base);
      l[h] = l[h] * alpha[h] + s;
      m[h] = mx;
    }
    const uint8_t* vp = a.v_cache + bh * kBlock * D;
    for (int i = tid; i < kBlock * D; i += kThreads) {
      const int64_t kpos = j * kBlock + i / D;
      kv[i / D * (D + 1) + i % D] = kpos >= lo && kpos < hi ? e4m3(vp[i]) : 0.f;
    }
    __syncthreads();
    const float vs = a.v_scale[bh];
    for (int i = tid; i < G * D; i += kThreads) {
      const int h = i / D, d = i % D;
      float s = 0.f;
      for (int k = 0; k < kBlock; ++k) s = fmaf(p[h * kBlock + k], kv[k * (D + 1) + d], s);
      acc[i] = acc[i] * alpha[h] + s * vs;
    }
    __syncthreads();
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((int64_t)t * a.H + (int64_t)g * G) * D;
  for (int i = tid; i < G * D; i += kThreads)
    out[i] = __float2bfloat16(l[i / D] > 0.f || l[i / D] != l[i / D] ? acc[i] / l[i / D] : 0.f);
  for (int h = tid; h < G; h += kThreads)
    a.lse[(int64_t)t * a.H + g * G + h] = l[h] == 0.f ? -INFINITY : m[h] + logf(l[h]);
}

}  // namespace

cudaError_t launch_paged_attention(const PagedAttnArgs& a, cudaStream_t stream) {
  const int G = a.H / a.HK;
  const size_t smem = sizeof(float) * ((size_t)2 * G * a.D + kBlock * (a.D + 1) + G * kBlock + 3 * G);
  auto kernel = a.D == 128 ? paged_attn_simple_kernel<128> : paged_attn_simple_kernel<64>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3((unsigned)a.T, (unsigned)a.HK), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace smla
