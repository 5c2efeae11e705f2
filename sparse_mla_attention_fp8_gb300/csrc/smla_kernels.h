// Internal launch interface between the C-ABI layer and the CUDA kernels.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace smla {

cudaError_t launch_quantize_store(const void* kv_new, const int64_t* slot_mapping, uint8_t* cache, int T, int64_t NB,
                                  cudaStream_t stream);

cudaError_t launch_translate(const int32_t* indices, const int32_t* block_table, const int32_t* req_id,
                             int32_t* slots, int T, int K, int R, int MB, int64_t NB, cudaStream_t stream);

// Separate-mode FP8 prefill: index translation with a prefill workspace, and
// the gather + up-convert of prefill requests' cache rows into a bf16 workspace.
cudaError_t launch_translate_ws(const int32_t* indices, const int32_t* block_table, const int32_t* req_id,
                                const int32_t* prefill_req_id, const int32_t* starts, int P, int32_t* out, int T,
                                int K, int R, int MB, int64_t NB, cudaStream_t stream);
cudaError_t launch_gather_upconvert(const uint8_t* cache, int64_t NB, const int32_t* block_table, int R, int MB,
                                    const int32_t* seq_lens, const int32_t* starts, void* ws, int64_t N,
                                    int num_sms, cudaStream_t stream);

// MLA weight absorption around the attention (smla_absorb.cu): per-head GEMMs
// on the tensor cores.  status: a device word that a timed-out wait sets.
cudaError_t launch_absorb_q(const void* q, const void* w_uk_t, void* q_out, int T, int H, int P, int* status,
                            cudaStream_t stream);
cudaError_t launch_v_up_proj(const void* attn_out, const void* w_uv, void* out, int T, int H, int V, int* status,
                             cudaStream_t stream);

// Work decomposition of one sparse-attention call: units are (token, head
// group) pairs, each split into nt tiles of 64 top-k rows; G persistent CTAs
// take contiguous, balanced ranges of the unit-major tile sequence.
struct AttnPlan {
  int HG;             // heads per work unit
  int n_hg;           // head groups per token
  int nt;             // tiles per unit
  int64_t units;      // T * n_hg
  int64_t total;      // units * nt
  int G;              // CTAs
  bool need_combine;  // some unit spans more than one CTA, merged by the combine kernel
  size_t ws_bytes;    // workspace bytes (status word + partial results)
  int cluster = 1;    // > 1: every unit is split into `cluster` parts run by one thread-block
                      // cluster, merged in distributed shared memory (no combine kernel)
  bool fused = false; // 128-head FP8 decode: every split unit has two parts, merged in the
                      // attention kernel by whichever part finishes second (no combine kernel)
};

AttnPlan plan_attention(bool fp8, int T, int H, int K, int num_splits, int num_sms);
AttnPlan plan_decode_fp8(int T, int H, int K, int num_splits, int num_sms);
AttnPlan plan_prefill_bf16(int T, int H, int K, int num_splits, int num_sms);

struct AttnArgs {
  const void* q;
  const uint8_t* cache;      // FP8 decode: [NB, 64, 656]
  const void* kv;            // BF16 prefill: [N, 576]
  const int32_t* indices;    // [T, K]
  const int32_t* block_table;
  const int32_t* req_id;
  void* out;                 // bf16 [T, H, 512]
  float* lse;                // [T, H]
  void* workspace;
  float sm_scale;
  int T, H, K, R, MB;
  int64_t NB;                // physical blocks (FP8) or kv rows (BF16)
};

cudaError_t launch_attention(bool fp8, const AttnArgs& a, const AttnPlan& plan, cudaStream_t stream);

// Attention with all 128 heads of a token per CTA pair (smla_wide.cu), over
// the bf16 latent buffer (prefill) or the FP8 paged cache (decode).
bool wide_supported(int H);
AttnPlan plan_prefill_wide(int T, int K, int num_splits, int num_sms);
AttnPlan plan_decode_wide(int T, int K, int num_splits, int num_sms);
cudaError_t launch_prefill_wide(const AttnArgs& a, const AttnPlan& plan, cudaStream_t stream);
cudaError_t launch_decode_wide(const AttnArgs& a, const AttnPlan& plan, cudaStream_t stream);
cudaError_t launch_decode_fp8(const AttnArgs& a, const AttnPlan& plan, cudaStream_t stream);

// The 128-head FP8 decode with the query quantized to e4m3 (two terms) and
// both products on the FP8 tensor path, the row scales folded into P
// (smla_wide8.cu).
AttnPlan plan_decode_wide8(int T, int K, int num_splits, int num_sms);
cudaError_t launch_decode_wide8(const AttnArgs& a, const AttnPlan& plan, cudaStream_t stream);
cudaError_t launch_prefill_bf16(const AttnArgs& a, const AttnPlan& plan, cudaStream_t stream);

// The NVFP4 cache (smla_nvfp4.cu): quantize-and-store, and the decode's
// staging of each token's top-k rows as exact bf16 rows ([T * K] row indices,
// -1 = invalid, then [T * K, 576] bf16 rows; nvfp4_stage_bytes in all).
cudaError_t launch_nvfp4_store(const void* kv_new, const int64_t* slot_mapping, uint8_t* cache, int T, int64_t NB,
                               cudaStream_t stream);
size_t nvfp4_stage_bytes(int T, int K);
cudaError_t launch_nvfp4_stage(const uint8_t* cache, int64_t NB, const int32_t* indices, const int32_t* block_table,
                               const int32_t* req_id, int T, int K, int R, int MB, void* stage, cudaStream_t stream);
// The native NVFP4 decode (smla_attn.cu) below 128 heads, in 16-head groups:
// a.cache is the NVFP4 cache, a.NB its blocks.
bool nvfp4_native_supported(int H);
AttnPlan plan_decode_nvfp4(int T, int H, int K, int num_splits, int num_sms);
cudaError_t launch_decode_nvfp4(const AttnArgs& a, const AttnPlan& plan, cudaStream_t stream);

// ---- paged K/V cache (block size 64, separate K and V heads)

// Requests of one batch: the block-table kernels keep their prefix sums over
// the requests in shared memory, one thread of an 8-CTA cluster per request.
constexpr int kMaxPagedRequests = 8192;

// Block tables, slot maps and token positions from request lengths
// (smla_blocks.cu).
struct BlocksExtendArgs {
  const int32_t* context_lens;  // [R]
  const int32_t* query_lens;    // [R]
  int32_t* block_table;         // [R, MB], new entries written
  const int32_t* free_blocks;   // [F] stack, top at free_count - 1
  const int32_t* free_count;    // [1]
  int32_t* query_start;         // [R + 1]
  int32_t* seq_lens;            // [R]
  int32_t* req_id_per_token;    // [T]
  int32_t* positions;           // [T]
  int64_t* slot_mapping;        // [T]
  int32_t* free_count_out;      // [1]
  int32_t* missing;             // [1]
  int R, MB, F, T;
  int64_t NB;
};
struct BlocksReleaseArgs {
  const uint8_t* release;      // [R], nonzero = release
  const int32_t* seq_lens;     // [R]
  const int32_t* block_table;  // [R, MB]
  int32_t* free_blocks;        // [F] stack
  const int32_t* free_count;   // [1]
  int32_t* context_lens;       // [R]
  int32_t* free_count_out;     // [1]
  int R, MB, F;
  int64_t NB;
  int chunk = 0;               // table entries per unit (set by the launch)
};
cudaError_t launch_blocks_extend(const BlocksExtendArgs& a, cudaStream_t stream);
cudaError_t launch_blocks_release(BlocksReleaseArgs a, cudaStream_t stream);

// Quantize-and-store of new K and V rows, a scale per block and head
// (smla_kvstore.cu).
struct KvStoreArgs {
  const void* k;               // bf16 [T, HK, D], rows k_stride elements apart
  const void* v;
  int64_t k_stride, v_stride;
  const int32_t* query_start;  // [R + 1]
  const int32_t* seq_lens;     // [R]
  const int32_t* block_table;  // [R, MB]
  uint8_t* k_cache;            // [NB, HK, 64, D]
  uint8_t* v_cache;
  float* k_scale;              // [NB, HK]
  float* v_scale;
  int T, HK, D, R, MB;
  int64_t NB;
};
cudaError_t launch_kv_store(const KvStoreArgs& a, cudaStream_t stream);

// Attention over the paged K/V cache (smla_paged_attn.cu).
struct PagedAttnArgs {
  const void* q;               // bf16 [T, H, D], rows q_stride elements apart
  int64_t q_stride;
  const uint8_t* k_cache;      // [NB, HK, 64, D]
  const uint8_t* v_cache;
  const float* k_scale;        // [NB, HK]
  const float* v_scale;
  const int32_t* block_table;  // [R, MB]
  const int32_t* seq_lens;     // [R]
  const int32_t* query_start;  // [R + 1]
  const float* alibi_slopes;   // [H] or null
  const int32_t* prefix_lens;  // [R] or null
  const int32_t* doc_start;    // [T] or null
  void* out;                   // bf16 [T, H, D]
  float* lse;                  // [T, H]
  void* workspace;
  float sm_scale, softcap;
  int window;
  int T, H, HK, D, R, MB;
  int64_t NB;
};
// Many rows per query tile (smla_paged_prefill.cu); called by launch_paged_attention.
size_t paged_prefill_workspace(int T, int H, int D, int R, int num_sms);
cudaError_t launch_paged_prefill(const PagedAttnArgs& a, int num_sms, cudaStream_t stream);
// max_query_len: an estimate.
size_t paged_attention_workspace(int T, int H, int HK, int D, int R, int max_query_len, int num_sms);
cudaError_t launch_paged_attention(const PagedAttnArgs& a, int max_query_len, int num_sms, cudaStream_t stream);
// The current device's words that a wait which ran out in the kernels of either file sets, and a kernel of each
// file whose only wait runs out.
cudaError_t paged_attn_timed_out(int** word);
cudaError_t paged_prefill_timed_out(int** word);
cudaError_t paged_attn_wait_check(int* status, cudaStream_t stream);
cudaError_t paged_prefill_wait_check(int* status, cudaStream_t stream);

// ---- MXFP8 operators: e4m3 codes with a scale exponent per 32 values

struct MxQuantizeArgs {
  const void* x;  // bf16 or float32 [T, K], rows x_stride elements apart
  int64_t x_stride;
  bool x_f32;
  uint8_t* codes;   // [T, K]
  uint8_t* scales;  // [T, K / 32], rows scale_stride bytes apart
  int64_t scale_stride;
  int T, K;
};
struct MxNormArgs {
  const void* x;         // bf16 [T, K], rows x_stride elements apart
  int64_t x_stride;
  const void* residual;  // the same, or null
  int64_t residual_stride;
  const void* weight;    // bf16 or float32 [K], or null
  bool weight_f32;
  float eps;
  uint8_t* codes;        // [T, K] or null
  uint8_t* scales;       // [T, K / 32], rows scale_stride bytes apart
  int64_t scale_stride;
  void* normed;          // bf16 [T, K] or null
  void* residual_out;    // bf16 [T, K] or null
  int T, K;
};
constexpr int kMaxNormK = 65536;  // a row is held in one CTA's registers
// (smla_mxnorm.cu)
cudaError_t launch_mx_quantize(const MxQuantizeArgs& a, cudaStream_t stream);
cudaError_t launch_mx_norm(const MxNormArgs& a, int num_sms, cudaStream_t stream);

// What a product's results go through and where they go.
struct MxEpilogue {
  const void* bias;      // bf16 or float32 [rows of W], or null
  bool bias_f32;
  int activation;        // SMLA_ACT_*
  const void* residual;  // bf16 [T, N], rows residual_stride elements apart, or null
  int64_t residual_stride;
  void* out;             // bf16 [T, N], or null where the results are quantized
  uint8_t* codes;        // [T, N]
  uint8_t* scales;       // [T, N / 32], rows scale_stride bytes apart
  int64_t scale_stride;
};
struct MxLinearArgs {
  const uint8_t* x;        // [T, K], rows x_stride bytes apart
  int64_t x_stride;
  const uint8_t* x_scale;  // [T, K / 32], rows x_scale_stride bytes apart
  int64_t x_scale_stride;
  const uint8_t* w;        // [N or 2 N, K]
  const uint8_t* w_scale;
  int64_t w_scale_stride;
  MxEpilogue to;
  int T, N, K;
  bool give_up;  // for tests: the kernels' waits run out at once
};
// (smla_linear.cu)
cudaError_t launch_mx_linear(const MxLinearArgs& a, int num_sms, cudaStream_t stream);
// The current device's word that a wait which ran out in the products' kernels sets, and a kernel whose only wait does.
cudaError_t mx_linear_timed_out(int** word);
cudaError_t mx_linear_wait_check(cudaStream_t stream);

struct MoeRouteArgs {
  const void* logits;  // bf16 or float32 [T, E]
  bool logits_f32;
  const float* bias;   // [E] or null
  bool sigmoid, renormalize;
  float scale;
  int groups, topk_groups;
  int32_t* ids;        // [T, topk]
  float* weights;      // [T, topk]
  int T, E, topk;
};
constexpr int kMaxRouteExperts = 512;
constexpr int kMaxTopk = 32;
// (smla_route.cu)
cudaError_t launch_moe_route(const MoeRouteArgs& a, cudaStream_t stream);

struct MoeArgs {
  const uint8_t* x;  // [T, K] as for the linear product
  int64_t x_stride;
  const uint8_t* x_scale;
  int64_t x_scale_stride;
  const int32_t* ids;    // [T, topk]
  const float* weights;  // [T, topk]
  const uint8_t* w13;    // [E, 2 F, K]
  const uint8_t* w13_scale;
  int64_t w13_scale_stride;
  const uint8_t* w2;     // [E, K, F]
  const uint8_t* w2_scale;
  int64_t w2_scale_stride;
  const void* residual;  // bf16 [T, K] or null
  int64_t residual_stride;
  void* out;             // bf16 [T, K]
  void* workspace;
  int T, E, topk, K, F;
  bool give_up;  // as for the linear product
};
// (smla_moe.cu)
size_t moe_workspace(int T, int E, int topk, int F);
cudaError_t launch_moe(const MoeArgs& a, int num_sms, cudaStream_t stream);
cudaError_t moe_timed_out(int** word);
cudaError_t moe_wait_check(cudaStream_t stream);

// Offsets inside the workspace.
constexpr size_t kWsStatusBytes = 256;

}  // namespace smla
