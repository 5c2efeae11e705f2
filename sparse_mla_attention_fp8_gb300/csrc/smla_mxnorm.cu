// Quantization to MXFP8, alone and behind the RMS norm with the residual's
// addition:  h = bf16(x + residual),  y = h / sqrt(mean h^2 + eps) * w,  and the
// codes and scales of y, from its float32 values.
//
// Both read and write each value once and are bound by HBM, for few rows by
// latency.  Four threads hold a group of 32 values (8 each, one 16-byte load of
// bf16), so a group's scale takes two shuffles.  The norm keeps its row in
// registers between the sum of squares and the output.
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

// The codes of 8 of a group's 32 values, its other 24 in the other lanes of this
// four (all of them active); the first of them writes the scale.
__device__ __forceinline__ void store_codes(const float (&v)[8], uint8_t* codes, uint8_t* scale) {
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, mx_finite_bits(v[i]));
  const uint32_t quad = 0xfu << (threadIdx.x & 28u);
  top = max(top, __shfl_xor_sync(quad, top, 1));
  top = max(top, __shfl_xor_sync(quad, top, 2));
  const int e = mx_exponent(top);
  const float inv = mx_pow2(-e);
  *reinterpret_cast<uint2*>(codes) = make_uint2(mx_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                                                mx_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
  if ((threadIdx.x & 3) == 0) *scale = (uint8_t)(e + 127);
}

constexpr int kQuantThreads = 256;

template <typename X>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const __grid_constant__ MxQuantizeArgs a) {
  grid_dependency_wait();
  const uint32_t per_row = (uint32_t)a.K / 8;
  const uint64_t i = (uint64_t)blockIdx.x * kQuantThreads + threadIdx.x;
  if (i >= (uint64_t)a.T * per_row) return;  // (a group's four threads go together)
  const uint32_t row = (uint32_t)(i / per_row), col = (uint32_t)(i - (uint64_t)row * per_row) * 8;
  float v[8];
  load8(static_cast<const X*>(a.x) + row * a.x_stride + col, v);
  store_codes(v, a.codes + (int64_t)row * a.K + col, a.scales + row * a.scale_stride + col / kMxGroup);
}

// One row by kWarps warps, kChunks groups of 8 values a thread; a CTA has
// kRows rows.
template <int kWarps, int kChunks, int kRows, typename W>
__global__ void __launch_bounds__(32 * kWarps * kRows) norm_kernel(const __grid_constant__ MxNormArgs a) {
  __shared__ float part[kRows][kWarps];
  constexpr int kThreads = 32 * kWarps;
  const int r = (int)threadIdx.x / kThreads, t = (int)threadIdx.x % kThreads;
  const int64_t row = (int64_t)blockIdx.x * kRows + r;
  const bool mine = row < a.T;
  grid_dependency_wait();
  uint4 h[kChunks];
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = 8 * (c * kThreads + t);
    h[c] = make_uint4(0u, 0u, 0u, 0u);
    if (!mine || col >= a.K) continue;
    float v[8];
    load8(static_cast<const __nv_bfloat16*>(a.x) + row * a.x_stride + col, v);
    if (a.residual) {
      float u[8];
      load8(static_cast<const __nv_bfloat16*>(a.residual) + row * a.residual_stride + col, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += u[i];
    }
    h[c] = pack8(v);
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = 8 * (c * kThreads + t);
    if (a.residual_out && mine && col < a.K)
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.residual_out) + row * a.K + col) = h[c];
    const uint32_t u[4] = {h[c].x, h[c].y, h[c].z, h[c].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = __uint_as_float(u[i] << 16), hi = __uint_as_float(u[i] & 0xffff0000u);
      sum = fmaf(lo, lo, fmaf(hi, hi, sum));
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
  if (kWarps > 1) {
    if ((t & 31) == 0) part[r][t >> 5] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += part[r][w];
  }
  if (!mine) return;
  const float f = rsqrtf(sum / (float)a.K + a.eps);
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = 8 * (c * kThreads + t);
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

template <typename W>
cudaError_t launch_norm(const MxNormArgs& a, cudaStream_t stream) {
  auto go = [&](auto kernel, int warps, int rows) {
    return launch(kernel, ((int64_t)a.T + rows - 1) / rows, 32 * warps * rows, stream, a);
  };
  if (a.K <= 256) return go(norm_kernel<1, 1, 8, W>, 1, 8);
  if (a.K <= 1024) return go(norm_kernel<4, 1, 2, W>, 4, 2);
  if (a.K <= 2048) return go(norm_kernel<8, 1, 1, W>, 8, 1);
  if (a.K <= 4096) return go(norm_kernel<16, 1, 1, W>, 16, 1);
  if (a.K <= 8192) return go(norm_kernel<16, 2, 1, W>, 16, 1);
  if (a.K <= 16384) return go(norm_kernel<16, 4, 1, W>, 16, 1);
  return go(norm_kernel<32, 8, 1, W>, 32, 1);
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantizeArgs& a, cudaStream_t stream) {
  const int64_t ctas = ((int64_t)a.T * (a.K / 8) + kQuantThreads - 1) / kQuantThreads;
  return a.x_f32 ? launch(quantize_kernel<float>, ctas, kQuantThreads, stream, a)
                 : launch(quantize_kernel<__nv_bfloat16>, ctas, kQuantThreads, stream, a);
}

cudaError_t launch_mx_norm(const MxNormArgs& a, cudaStream_t stream) {
  return a.weight_f32 ? launch_norm<float>(a, stream) : launch_norm<__nv_bfloat16>(a, stream);
}

}  // namespace smla
