// Quantization to MXFP8, alone and behind the RMS norm with the residual's
// addition:  h = bf16(x + residual),  y = h / sqrt(mean h^2 + eps) * w,  and the
// codes and scales of y, from its float32 values.
//
// Both read and write each value once and are bound by HBM, for few rows by
// latency.  Four threads hold a group of 32 values (8 each, one 16-byte load of
// bf16), in the quantization two, so a group's scale takes one or two shuffles.  The
// norm keeps its row in registers between the sum of squares and the output.
// Measured: 11264 x 4096 weights (140 MB) quantized in 24.3 us, 5.8 TB/s with the
// launch (with 8 values a thread, and their 64-bit divisions, 31); 7000 x 5120 with
// residual and bf16 norm (324 MB) 56.8 us, 5.7 TB/s; one row of 4096 2.1 us.
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sm103_ptx.cuh"
#include "smla_common.cuh"
#include "smla_kernels.h"
#include "smla_mxfp8.cuh"

namespace smla {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// The scale's exponent of a group of 32 values, kCount of them here and the others in the other lanes of these
// 32 / kCount (all of them active).
template <int kCount>
__device__ __forceinline__ int group_exponent(const float (&v)[kCount]) {
  constexpr int kLanes = 32 / kCount;
  const uint32_t lanes = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < kCount; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
  for (int d = 1; d < kLanes; d *= 2) top = max(top, __shfl_xor_sync(lanes, top, d));
  if (top >= 0x7f800000u) {  // infinities and NaN are left out
    top = 0u;
#pragma unroll
    for (int i = 0; i < kCount; ++i) top = max(top, mx_finite_bits(v[i]));
#pragma unroll
    for (int d = 1; d < kLanes; d *= 2) top = max(top, __shfl_xor_sync(lanes, top, d));
  }
  return mx_exponent(top);
}

// The codes of 8 of a group's values; the first of its four threads writes the scale.
__device__ __forceinline__ void store_codes(const float (&v)[8], uint8_t* codes, uint8_t* scale) {
  const int e = group_exponent(v);
  const float inv = mx_pow2(-e);
  *reinterpret_cast<uint2*>(codes) = make_uint2(mx_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                                                mx_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
  if ((threadIdx.x & 3) == 0) *scale = (uint8_t)(e + 127);
}

constexpr int kQuantThreads = 256;

// 16 values a thread, two threads a group.
template <typename X>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const __grid_constant__ MxQuantizeArgs a) {
  grid_dependency_wait();
  const uint32_t per_row = (uint32_t)a.K / 16, count = (uint32_t)a.T * per_row;  // (below 2^32 by the launch)
  const uint32_t i = blockIdx.x * kQuantThreads + threadIdx.x;
  if (i >= count) return;  // (a group's two threads go together)
  const uint32_t row = i / per_row, col = (i - row * per_row) * 16;
  const X* x = static_cast<const X*>(a.x) + row * a.x_stride + col;
  float lo[8], hi[8], v[16];
  load8(x, lo);
  load8(x + 8, hi);
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = lo[k], v[8 + k] = hi[k];
  const int e = group_exponent(v);
  const float inv = mx_pow2(-e);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = mx_e4m3x4(v[4 * k] * inv, v[4 * k + 1] * inv, v[4 * k + 2] * inv, v[4 * k + 3] * inv);
  *reinterpret_cast<uint4*>(a.codes + (int64_t)row * a.K + col) = make_uint4(w[0], w[1], w[2], w[3]);
  if ((threadIdx.x & 1) == 0) a.scales[row * a.scale_stride + col / kMxGroup] = (uint8_t)(e + 127);
}

// Rows by CTAs of whole warps, kChunks groups of 8 values a thread.  A CTA takes every gridDim-th row and (where
// registers allow) loads the next one before it has the sum of the present one.
template <int kChunks, typename W>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ MxNormArgs a) {
  constexpr bool kAhead = kChunks <= 2;
  __shared__ float part[2][32];
  const int t = (int)threadIdx.x, threads = (int)blockDim.x, warps = threads / 32;
  const int col0 = 8 * t;
  grid_dependency_wait();
  uint4 x[kAhead ? kChunks : 1], r[kAhead ? kChunks : 1];
  // (plain loads: the sum may go back to where x or the residual lies)
  auto load = [&](int64_t row, int c, uint4& x, uint4& r) {
    const int col = col0 + 8 * threads * c;
    x = r = make_uint4(0u, 0u, 0u, 0u);
    if (row >= a.T || col >= a.K) return;
    x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + row * a.x_stride + col);
    if (a.residual)
      r = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.residual) + row * a.residual_stride + col);
  };
  if (kAhead)
#pragma unroll
    for (int c = 0; c < kChunks; ++c) load(blockIdx.x, c, x[c], r[c]);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
    uint4 h[kChunks];
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int k = kAhead ? c : 0;
      if (!kAhead) load(row, c, x[k], r[k]);
      const uint32_t u[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, v[4] = {r[k].x, r[k].y, r[k].z, r[k].w};
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = u[i];
        if (a.residual)
          w[i] = pack_bf16x2(__uint_as_float(u[i] << 16) + __uint_as_float(v[i] << 16),
                             __uint_as_float(u[i] & 0xffff0000u) + __uint_as_float(v[i] & 0xffff0000u));
        const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
        sum = fmaf(lo, lo, fmaf(hi, hi, sum));
      }
      h[c] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (kAhead)
#pragma unroll
      for (int c = 0; c < kChunks; ++c) load(row + gridDim.x, c, x[c], r[c]);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int col = col0 + 8 * threads * c;
      if (a.residual_out && col < a.K)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.residual_out) + row * a.K + col) = h[c];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    if (warps > 1) {
      if ((t & 31) == 0) part[turn][t >> 5] = sum;
      __syncthreads();
      sum = (t & 31) < warps ? part[turn][t & 31] : 0.f;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    }
    const float f = rsqrtf(sum / (float)a.K + a.eps);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int col = col0 + 8 * threads * c;
      if (col >= a.K) break;
      float y[8];
      const uint32_t u[4] = {h[c].x, h[c].y, h[c].z, h[c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = __uint_as_float(u[i] << 16) * f;
        y[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u) * f;
      }
      if (a.weight) {
        float w[8];
        load8(static_cast<const W*>(a.weight) + col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= w[i];
      }
      if (a.normed) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.normed) + row * a.K + col) = pack8(y);
      if (a.codes) store_codes(y, a.codes + row * a.K + col, a.scales + row * a.scale_stride + col / kMxGroup);
    }
  }
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int64_t ctas, int threads, cudaStream_t stream, const Args&... args) {
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// As many CTAs as the SMs hold at once (by their registers: 64 a thread).
template <int kChunks, typename W>
cudaError_t launch_rows(const MxNormArgs& a, int num_sms, cudaStream_t stream) {
  const int threads = (a.K / 8 + kChunks * 32 - 1) / (kChunks * 32) * 32;
  const int64_t ctas = std::min<int64_t>(a.T, (int64_t)num_sms * std::min(32, 1024 / threads));
  return launch(norm_kernel<kChunks, W>, ctas, threads, stream, a);
}
template <typename W>
cudaError_t launch_norm(const MxNormArgs& a, int num_sms, cudaStream_t stream) {
  // For many rows two groups a thread: more rows are in flight on an SM (7000 x 5120 without the bf16 norm 40.9 us, with
  // one group 53.0; 400 x 4096 3.6 and 3.8; one row is better off with one).
  const bool many = a.T > 2 * num_sms;
  if (a.K <= 8 * 1024) return many ? launch_rows<2, W>(a, num_sms, stream) : launch_rows<1, W>(a, num_sms, stream);
  if (a.K <= 16 * 1024) return launch_rows<2, W>(a, num_sms, stream);
  if (a.K <= 32 * 1024) return launch_rows<4, W>(a, num_sms, stream);
  return launch_rows<8, W>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantizeArgs& all, cudaStream_t stream) {
  MxQuantizeArgs a = all;
  const int64_t most = (int64_t{1} << 31) / (a.K / 16) - 1;  // rows a launch
  cudaError_t e = cudaSuccess;
  for (int64_t done = 0; done < all.T && e == cudaSuccess; done += a.T) {
    a.T = (int)std::min<int64_t>(most, all.T - done);
    a.x = static_cast<const char*>(all.x) + done * all.x_stride * (all.x_f32 ? 4 : 2);
    a.codes = all.codes + done * all.K;
    a.scales = all.scales + done * all.scale_stride;
    const int64_t ctas = ((int64_t)a.T * (a.K / 16) + kQuantThreads - 1) / kQuantThreads;
    e = a.x_f32 ? launch(quantize_kernel<float>, ctas, kQuantThreads, stream, a)
                : launch(quantize_kernel<__nv_bfloat16>, ctas, kQuantThreads, stream, a);
  }
  return e;
}

cudaError_t launch_mx_norm(const MxNormArgs& a, int num_sms, cudaStream_t stream) {
  return a.weight_f32 ? launch_norm<float>(a, num_sms, stream) : launch_norm<__nv_bfloat16>(a, num_sms, stream);
}

}  // namespace smla
