// Linear product on MXFP8 operands with its epilogue: y = act(x W^T + b) +
// residual, or silu(x Wg^T + bg) * (x Wu^T + bu), in bf16 or MXFP8.
#include "smla_mxgemm.cuh"
#include "smla_mxpair.cuh"

namespace smla {

namespace {

template <int MODE, int NT>
cudaError_t launch_tiles(const MxLinearArgs& a, const MxParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kGate = MODE == kGated ? 2 : 1;
  CUtensorMap a_map, b_map;
  cudaError_t e = code_map(&a_map, a.w, (int64_t)kGate * a.N, a.K, a.K, kTileRows / kGate);
  if (e == cudaSuccess) e = code_map(&b_map, a.x, a.T, a.K, a.x_stride, NT);
  if (e != cudaSuccess) return e;
  const int64_t rows = ((int64_t)a.N * kGate + kTileRows - 1) / kTileRows, tokens = ((int64_t)a.T + NT - 1) / NT;
  const int parts = split_k(rows * tokens, (a.K + kStepK - 1) / kStepK, num_sms);
  return launch_mx<MODE, NT>(p, parts, rows, tokens, 1, a_map, b_map, stream);
}
template <int MODE>
cudaError_t launch_few(const MxLinearArgs& a, const MxParams& p, int num_sms, cudaStream_t stream) {
  if (a.T <= 16) return launch_tiles<MODE, 16>(a, p, num_sms, stream);
  if (a.T <= 32) return launch_tiles<MODE, 32>(a, p, num_sms, stream);
  if (a.T <= 64) return launch_tiles<MODE, 64>(a, p, num_sms, stream);
  return launch_tiles<MODE, 128>(a, p, num_sms, stream);
}

}  // namespace

cudaError_t launch_mx_linear(const MxLinearArgs& a, int num_sms, cudaStream_t stream) {
  MxParams p{};
  p.a_scale = a.w_scale;
  p.a_scale_stride = a.w_scale_stride;
  p.b_scale = a.x_scale;
  p.b_scale_stride = a.x_scale_stride;
  p.rows = a.N;
  p.T = a.T;
  p.K = a.K;
  p.give_up = a.give_up;
  p.to = a.to;
  p.ld = a.N;
  const auto even = [](const void* q, int64_t stride) { return stride % 2 == 0 && reinterpret_cast<uintptr_t>(q) % 4 == 0; };
  p.pairs = even(a.to.out, a.N) && (!a.to.residual || even(a.to.residual, a.to.residual_stride));
  // Rows of the latent cache's tokens and of its queries: mla_cache_store_fp8 and sparse_mla_decode_fp8 read these before they
  // wait for this grid, and begin once its CTAs have ended.  (The fence behind the results takes 0.4 us of a token's 6.0.)
  p.publish = a.to.out != nullptr && a.N % kDqk == 0;
  p.wide_scales = rows16(a.x_scale, a.x_scale_stride) && rows16(a.w_scale, a.w_scale_stride);
  // Pairs of CTAs where they have enough tiles, 24, or 8 with a short K.  Pairs | the other kernel: K = N = 4096: 16 tiles
  // (256 tokens) 12.8 | 12.3 us, 32 (400) 13.6 | 16.9; K = 8192, N = 1024: 12 tiles (700) 19.9 | 15.1, 24 (1500) 20.7 |
  // 22.2; K = N = 2048: 8 tiles (128) 8.7 | 9.9, 24 (700) 9.3 | 12.7.  Up to 64 tokens the other kernel's tiles have
  // fewer columns.
  const int64_t columns = a.to.activation == SMLA_ACT_SWIGLU ? 128 : 256;
  const int64_t pair_tiles = ((int64_t)a.N + 255) / 256 * ((a.T + columns - 1) / columns);
  if (a.T > 64 && pair_tiles >= (a.K <= 2048 ? 8 : 24)) {
    switch (a.to.activation) {
      case SMLA_ACT_NONE: return launch_pair<SMLA_ACT_NONE>(a, p, num_sms, stream);
      case SMLA_ACT_RELU: return launch_pair<SMLA_ACT_RELU>(a, p, num_sms, stream);
      case SMLA_ACT_SILU: return launch_pair<SMLA_ACT_SILU>(a, p, num_sms, stream);
      case SMLA_ACT_GELU: return launch_pair<SMLA_ACT_GELU>(a, p, num_sms, stream);
      case SMLA_ACT_GELU_TANH: return launch_pair<SMLA_ACT_GELU_TANH>(a, p, num_sms, stream);
      default: return launch_pair<SMLA_ACT_SWIGLU>(a, p, num_sms, stream);
    }
  }
  switch (a.to.activation) {
    case SMLA_ACT_SWIGLU: return launch_few<kGated>(a, p, num_sms, stream);
    case SMLA_ACT_GELU: return launch_few<kGelu>(a, p, num_sms, stream);
    default: return launch_few<kLinear>(a, p, num_sms, stream);
  }
}

cudaError_t mx_linear_wait_check(cudaStream_t stream) { return mx_wait_check(stream); }
cudaError_t mx_linear_timed_out(int** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_mx_timed_out); }

}  // namespace smla
