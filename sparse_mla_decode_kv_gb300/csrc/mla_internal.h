// Host-side declarations shared between the C-ABI layer (mla_api.cu) and the
// kernel translation units.  Not part of the public interface.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mla {

// Multiprocessor count of the current device (cached per device).
int device_sm_count();
// Device address of the library's fault word on the current device.
unsigned int* fault_word_ptr();
// Raises a kernel's dynamic shared-memory limit to `bytes` once per device:
// bit d of `*done` records device d (devices past 63 are configured on every
// call).  Safe when host threads drive different devices at once.
cudaError_t set_smem_limit_once(const void* kernel, int bytes, std::atomic<uint64_t>* done);
// True when the driver's tensor-map encoder is available (TMA paths need it).
bool tensor_maps_available();
// A 2-D TMA tensor map (no interleave, zero fill out of bounds) over `rows`
// rows of `inner` elements, rows `row_stride` bytes apart; box
// {box_inner, box_rows}.  False when the driver entry point is unavailable
// or the description is rejected.
bool encode_tensor_map_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t inner,
                          uint64_t rows, uint64_t row_stride, uint32_t box_inner, uint32_t box_rows,
                          CUtensorMapSwizzle swizzle);

// The same over bf16 values [rows][heads][inner] with strides of the two outer axes
// in bytes (not used for an axis of one entry); box 64 x box_heads x box_rows, the
// 128-byte swizzle.
bool encode_tensor_map_3d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t heads, uint64_t rows,
                          uint64_t head_stride, uint64_t row_stride, uint32_t box_heads, uint32_t box_rows);

cudaError_t launch_quantize_append(const uint16_t* latent, const uint16_t* rope, const int64_t* slot_mapping,
                                   int64_t n_tokens, void* pool, int64_t num_blocks, int64_t block_stride, int fmt,
                                   cudaStream_t stream);

cudaError_t launch_index_key_append(const uint16_t* keys, const int64_t* slot_mapping, int64_t n_tokens, void* pool,
                                    int64_t num_blocks, int64_t block_stride, cudaStream_t stream);

// Staged path: NVFP4 rows re-stored as FP8 rows (staged_bt / staged_ctx may be
// null; when given, the identity block table and context lengths are written).
cudaError_t launch_stage_rows_fp8(const void* pool, int64_t block_stride, int64_t num_blocks,
                                  const int32_t* block_table, int max_blocks_per_req, const int32_t* context_lens,
                                  const int32_t* topk_idx, int batch, int topk, void* staged, int32_t* staged_topk,
                                  int32_t* staged_bt, int32_t* staged_ctx, cudaStream_t stream);

// Sparse decode: split plan and launch.  The plan is made for the number of
// (request, query token) pairs; q_len query tokens per request share its
// block table and context (token i sees t < ctx - (q_len - 1 - i)).
struct DecodePlan {
  int splits;          // CTAs per (request, 16-head group) along the top-k list
  int rows_per_split;  // multiple of 16
  bool cluster;        // the splits form a thread-block cluster and merge through DSMEM
  size_t workspace;    // bytes of split partials in global memory (0 for one split or a cluster merge)
};
DecodePlan plan_sparse_decode(int batch, int num_heads, int topk);
cudaError_t launch_sparse_decode(int fmt, const uint16_t* q_nope, const uint16_t* q_rope, const void* pool,
                                 int64_t block_stride, int64_t num_blocks, const int32_t* block_table,
                                 int max_blocks_per_req, const int32_t* context_lens, const int32_t* topk_idx,
                                 int batch, int q_len, int num_heads, int topk, float softmax_scale, uint16_t* out,
                                 float* lse, void* workspace, const DecodePlan& plan, cudaStream_t stream);

// Tensor-memory decode for 64-head blocks of NVFP4 rows in a pool TMA can
// gather from (sparse_decode_tc.cu).  Split partials use the workspace
// layout of the 16-head kernel.
struct TcDecodeParams {
  const uint16_t* q_nope;
  const uint16_t* q_rope;
  int64_t block_stride;
  int64_t num_blocks;
  const int32_t* block_table;
  int max_blocks_per_req;
  const int32_t* context_lens;
  const int32_t* topk_idx;
  int pairs;
  int q_len;
  int num_heads;
  int topk;
  int splits;
  float softmax_scale;
  uint16_t* out;
  float* lse;
  void* part_o;
  float* part_lse;
  unsigned int* fault_word;
};
bool sparse_decode_tc_supported(int fmt, int num_heads);
// The call runs the tensor-memory kernel (format, head count and a pool TMA
// can describe as a tensor of 352-byte rows; the pool base must also be
// 16-byte aligned, which every entry point already requires).
bool sparse_decode_uses_tc(int fmt, int num_heads, int64_t block_stride, int64_t num_blocks);
int plan_sparse_decode_tc(int pairs, int num_heads, int topk, int max_splits);
cudaError_t launch_sparse_decode_tc(const TcDecodeParams& p, const CUtensorMap& map, cudaStream_t stream);

// Dense decode over a window and / or a shared prefix (dense_decode.cu).
struct DensePlan {
  int groups_per_req;  // 64-column groups of a request's (query token, head) pairs
  int splits;          // CTAs per group along its own rows
  int prefix_groups;   // 64-column groups of the whole batch over the prefix (0 without one)
  int prefix_splits;   // CTAs per such group along the prefix
  size_t workspace;    // bytes of partials, 0 for a single slice
};
struct DenseArgs {
  const uint16_t* q_nope;
  const uint16_t* q_rope;
  const uint8_t* pool;
  int64_t block_stride;
  int64_t num_blocks;
  const int32_t* prefix_table;
  int prefix_len;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* ctx_lens;
  int max_context;  // longer contexts are cut to it
  int batch;
  int q_len;
  int num_heads;
  int sinks;
  int window;
  float scale_log2;
  uint16_t* out;
  float* lse;
  // set by the launch from the plan
  int groups_per_req, splits, prefix_groups, prefix_splits, parts;
  int64_t columns;
  float* part_o;
  float* part_lse;
  unsigned int* fault_word;
};
DensePlan plan_dense_decode(int batch, int q_len, int num_heads, int64_t own_rows, int prefix_len);
cudaError_t launch_dense_decode(int fmt, DenseArgs a, const DensePlan& plan, void* workspace, cudaStream_t stream);

// Block tables and slot maps from request lengths (block_table.cu).
struct ExtendArgs {
  const int32_t* context_lens;
  const int32_t* new_lens;
  int batch;
  int32_t* block_table;
  int max_blocks;
  const int32_t* free_blocks;
  int64_t free_capacity;
  const int64_t* free_state;
  int64_t num_blocks;
  int64_t* slot_mapping;
  int32_t* positions;
  int64_t num_slots;
  int32_t* query_start;
  int32_t* context_lens_out;
  int64_t* free_state_out;
};
cudaError_t launch_block_table_extend(const ExtendArgs& a, cudaStream_t stream);

// Norms and rotation of query / key heads and of latent rows (norm_rope.cu).
struct HeadSet {  // bf16 heads [tokens, heads, dim], the last axis contiguous; null = none
  const uint16_t* in;
  uint16_t* out;
  int heads;
  int64_t in_token, in_head, out_token, out_head;  // strides in elements
  const uint16_t* weight;                          // bf16 [dim], or null: no norm
};
struct NormRopeArgs {
  HeadSet set[2];  // queries, keys
  int64_t tokens;
  int dim;
  int rope_offset;
  float eps;
  const int32_t* positions;
  const double* inv_freq;  // [32]
  bool interleaved;
  // latent rows into the cache
  const uint16_t* kv;  // bf16 [tokens, 576], or null
  int64_t kv_token;    // stride in elements
  const uint16_t* latent_weight;
  const int64_t* slot_mapping;
  uint8_t* pool;
  int64_t num_blocks;
  int64_t block_stride;
  int fmt;
};
cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream);

// Attention over packed prompts (prompt_attention.cu).
enum PromptVariant { kPromptPlain, kPromptTurns, kPromptPairs };
struct PromptPlan {
  int64_t places;    // of units, per key head
  int unit_tiles;    // tiles of rows in a unit: 1 or 2
  int splits;        // CTAs per pair along the keys
  PromptVariant variant;
  size_t workspace;  // bytes of partials, 0 for a single slice
};
struct PromptArgs {
  const uint16_t* q;  // bf16 [q_tokens, heads, dk], strides in elements
  const uint16_t* k;  // [kv_tokens, kv_heads, dk]
  const uint16_t* v;  // [kv_tokens, kv_heads, dv]
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  int q_tokens, kv_tokens;
  int batch;
  const int32_t* q_start;   // [batch + 1]
  const int32_t* kv_start;  // [batch + 1]
  int heads, kv_heads, dk, dv;
  bool causal;
  bool negate;       // a negative scale: the products are negated
  float scale_log2;  // > 0
  uint16_t* out;     // [q_tokens, heads, dv], strides in elements
  int64_t out_token, out_head;
  float* lse;  // [q_tokens, heads] or null
  // set by the launch from the plan
  int group, splits, places, unit_tiles;
  bool out_wide;  // rows of out begin and end at multiples of 32 bytes
  float* part_o;     // [q_tokens, heads, splits, dv]
  float2* part_lse;  // [q_tokens, heads, splits]: reference, log2 of the sum x 2^8 relative to it
  unsigned int* fault_word;
};
PromptPlan plan_prompt_attention(int64_t q_tokens, int64_t kv_tokens, int batch, int heads, int kv_heads, int dv);
// *described: whether the tensors' strides can be described to the copy engine; nothing
// is launched if not.
cudaError_t launch_prompt_attention(PromptArgs a, const PromptPlan& plan, void* workspace, cudaStream_t stream,
                                    bool* described);

// Residual's addition, norm and e4m3 output (add_norm_quant.cu).
struct AddNormArgs {
  const uint16_t* x;
  int64_t x_stride;  // elements, as the others
  int residual_type;  // 0 none, 1 bf16, 2 float
  const void* residual;
  int64_t res_stride;
  void* residual_out;
  int64_t res_out_stride;
  const uint16_t* weight;
  int64_t tokens;
  int dim;
  int group;         // 128, or 0: the row
  int scale_groups;  // scales per row
  float eps;
  float inv_dim;
  uint8_t* codes;  // [tokens, dim]
  float* scales;   // [tokens, scale_groups]
};
cudaError_t launch_add_norm_quant(const AddNormArgs& a, cudaStream_t stream);

// Products with 4-bit weights (fp4_matvec.cu).
struct MatvecArgs {
  const void* x;  // bf16, or e4m3 codes
  bool x_codes;
  int64_t x_token, x_group;  // strides in elements
  const float* x_scales;     // [tokens, groups, x_scale_groups], codes only
  int x_scale_groups;        // 1 or ceil(k / 128)
  const uint8_t* codes;      // [groups, n, k / 2]
  const uint8_t* scales;     // [groups, n, k / 16]
  const float* weight_scale;  // [groups] or null
  int64_t tokens;
  int groups;
  int n;
  int k;
  void* out;
  bool out_float;
  int64_t out_token, out_group;
  // set by the launch
  int row_warps_bits, splits, rows, slice, stage, smem;
};
cudaError_t launch_fp4_matvec(MatvecArgs a, cudaStream_t stream);

// Indexer and top-k.
size_t topk_workspace_bytes(int batch, int max_context_len, int topk);
cudaError_t launch_topk(const float* scores, int64_t row_stride, const int32_t* context_lens, int batch, int topk,
                        int max_context_len, int32_t* out, void* workspace, cudaStream_t stream);
cudaError_t launch_indexer_scores(const uint16_t* q_idx, const float* head_w, const void* key_pool,
                                  int64_t block_stride, int64_t num_blocks, const int32_t* block_table,
                                  int max_blocks_per_req, const int32_t* context_lens, int batch, int n_heads,
                                  int max_context_len, float* scores, int64_t scores_stride, cudaStream_t stream);

}  // namespace mla
