// Mixture of experts for few tokens, in two products: per expert the gated one,
// whose results, weighted by the token's weight for the expert, are quantized
// (h), then the down projection, whose reduction runs over the features of all
// of a tile's experts at once, so that the experts' results are summed in the
// accumulator.  Tokens are columns: an expert's weights are read once for all of
// them (columns of tokens that it does not have hold zeros), and a few columns
// more cost little beside that read, which bounds both products.  The second one is
// launched while the first runs and copies its first weights meanwhile.
//
// Measured, 64 experts of 3 x 4096 x 1024, 8 a token: one token 25.3 us (104 MB;
// the first product's last CTA ends after 15.4 us, the second's after 24.5), 48 tokens
// 143 to 146 us (805 MB, 5.5 TB/s).  The one token is bound by what follows one another:
// ids, weights, sums of a cluster, the launch's dependency, h, sums.
#include "smla_mxgemm.cuh"

namespace smla {

namespace {

int token_tile(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128; }

// behind the status word h: [token tile][expert slot][token][F] codes, then the scales, in rows on 16-byte boundaries
struct MoeSizes {
  int tile, slots;
  int64_t tiles, rows, scale_stride;
  size_t codes, scales, bytes;
};
MoeSizes moe_sizes(int T, int E, int topk, int F) {
  MoeSizes s;
  s.tile = token_tile(T);
  s.tiles = ((int64_t)T + s.tile - 1) / s.tile;
  s.slots = (int)std::min<int64_t>(E, (int64_t)std::min(T, s.tile) * topk);
  s.rows = s.tiles * s.slots * s.tile;
  s.scale_stride = (F / kMxGroup + 15) / 16 * 16;
  s.codes = kWsStatusBytes;
  s.scales = s.codes + ((size_t)s.rows * F + 255) / 256 * 256;
  s.bytes = s.scales + ((size_t)s.rows * s.scale_stride + 255) / 256 * 256;
  return s;
}

template <int NT>
cudaError_t launch_experts(const MoeArgs& a, const MoeSizes& s, int num_sms, cudaStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  MxParams up{}, down{};
  up.a_scale = a.w13_scale;
  up.a_scale_stride = a.w13_scale_stride;
  up.b_scale = a.x_scale;
  up.b_scale_stride = a.x_scale_stride;
  up.wide_scales = rows16(a.x_scale, a.x_scale_stride) && rows16(a.w13_scale, a.w13_scale_stride);
  up.rows = a.F;
  up.T = a.T;
  up.K = a.K;
  up.give_up = a.give_up;
  up.status = reinterpret_cast<int*>(ws);
  up.to.codes = ws + s.codes;
  up.to.scales = ws + s.scales;
  up.to.scale_stride = s.scale_stride;
  up.ld = a.F;
  up.ids = a.ids;
  up.weights = a.weights;
  up.topk = a.topk;
  up.E = a.E;
  up.slots = s.slots;
  down = up;
  down.a_scale = a.w2_scale;
  down.a_scale_stride = a.w2_scale_stride;
  down.b_scale = ws + s.scales;
  down.b_scale_stride = s.scale_stride;
  down.wide_scales = rows16(a.w2_scale, a.w2_scale_stride);
  down.rows = a.K;
  down.K = a.F;
  down.to = MxEpilogue{};
  down.to.out = a.out;
  down.to.residual = a.residual;
  down.to.residual_stride = a.residual_stride;
  down.ld = a.K;
  down.pairs = reinterpret_cast<uintptr_t>(a.out) % 4 == 0 && (!a.residual || (a.residual_stride % 2 == 0 &&
                                                                reinterpret_cast<uintptr_t>(a.residual) % 4 == 0));
  CUtensorMap w13, x, w2, h;
  cudaError_t e = code_map(&w13, a.w13, (int64_t)a.E * 2 * a.F, a.K, a.K, kTileRows / 2);
  if (e == cudaSuccess) e = code_map(&x, a.x, a.T, a.K, a.x_stride, NT);
  if (e == cudaSuccess) e = code_map(&w2, a.w2, (int64_t)a.E * a.K, a.F, a.F, kTileRows);
  if (e == cudaSuccess) e = code_map(&h, ws + s.codes, s.rows, a.F, a.F, NT);
  if (e != cudaSuccess) return e;
  const int64_t f_tiles = ((int64_t)2 * a.F + kTileRows - 1) / kTileRows, k_tiles = (a.K + kTileRows - 1) / kTileRows;
  const int up_parts = split_k(f_tiles * s.slots * s.tiles, (a.K + kStepK - 1) / kStepK, num_sms);
  e = launch_mx<kMoeUp, NT>(up, up_parts, f_tiles, s.tiles, s.slots, w13, x, stream);
  if (e != cudaSuccess) return e;
  const int down_parts = split_k(k_tiles * s.tiles, (int64_t)s.slots * ((a.F + kStepK - 1) / kStepK), num_sms);
  return launch_mx<kMoeDown, NT>(down, down_parts, k_tiles, s.tiles, 1, w2, h, stream);
}

}  // namespace

size_t moe_workspace(int T, int E, int topk, int F) { return moe_sizes(T, E, topk, F).bytes; }

cudaError_t launch_moe(const MoeArgs& a, int num_sms, cudaStream_t stream) {
  const MoeSizes s = moe_sizes(a.T, a.E, a.topk, a.F);
  if (s.rows > INT32_MAX) return cudaErrorInvalidValue;
  switch (s.tile) {
    case 16: return launch_experts<16>(a, s, num_sms, stream);
    case 32: return launch_experts<32>(a, s, num_sms, stream);
    case 64: return launch_experts<64>(a, s, num_sms, stream);
    default: return launch_experts<128>(a, s, num_sms, stream);
  }
}

cudaError_t moe_wait_check(cudaStream_t stream) { return mx_wait_check(stream); }
cudaError_t moe_timed_out(int** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_mx_timed_out); }

}  // namespace smla
