// The C ABI of libmla_nvfp4.so (declared in include/mla_nvfp4.h): host-side
// argument validation, workspace sizing and kernel dispatch.  Nothing here
// allocates device memory; every launch goes to the caller's stream.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

#include "../../include/mla_nvfp4.h"
#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {

// Set by bounded device waits that run out (bits in mla_device.cuh); read and
// cleared through mla_device_fault().
__device__ unsigned int g_fault_word = 0;

namespace {

thread_local int t_last_cuda_error = 0;

mla_status_t cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MLA_OK;
  t_last_cuda_error = static_cast<int>(e);
  return MLA_ERR_CUDA;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// block_size: 64 is supported; other powers of two are valid but unsupported.
mla_status_t check_block_size(int block_size) {
  if (block_size <= 0 || (block_size & (block_size - 1)) != 0) return MLA_ERR_INVALID_ARG;
  return block_size == kBlock ? MLA_OK : MLA_ERR_UNSUPPORTED;
}

int row_bytes(int fmt) { return fmt == MLA_KV_NVFP4 ? kRowNvfp4 : fmt == MLA_KV_FP8 ? kRowFp8 : 0; }

mla_status_t check_decode_args(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                               int64_t kv_block_stride, int64_t num_blocks, const int32_t* block_table,
                               int max_blocks_per_req, const int32_t* context_lens, const int32_t* topk_idx,
                               int batch, int num_heads, int block_size, int topk, float softmax_scale,
                               const uint16_t* out, int fmt) {
  if (batch < 0) return MLA_ERR_INVALID_ARG;
  mla_status_t s = check_block_size(block_size);
  if (s != MLA_OK) return s;
  if (num_heads < 16 || num_heads > 128 || num_heads % 16 != 0) return MLA_ERR_INVALID_ARG;
  if (topk < 1 || topk > 2048) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale)) return MLA_ERR_INVALID_ARG;
  if (batch == 0) return MLA_OK;
  if (!q_nope || !q_rope || !kv_pool || !block_table || !context_lens || !topk_idx || !out)
    return MLA_ERR_INVALID_ARG;
  if (!aligned(q_nope, 16) || !aligned(q_rope, 8) || !aligned(kv_pool, 16) || !aligned(out, 16) ||
      !aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(topk_idx, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_blocks < 0 || max_blocks_per_req < 1) return MLA_ERR_INVALID_ARG;
  if (kv_block_stride % 16 != 0 || kv_block_stride < static_cast<int64_t>(block_size) * row_bytes(fmt))
    return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

constexpr int kMaxQueryTokens = 64;

mla_status_t decode_impl(int fmt, const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                         int64_t kv_block_stride, int64_t num_blocks, const int32_t* block_table,
                         int max_blocks_per_req, const int32_t* context_lens, const int32_t* topk_idx, int batch,
                         int q_len, int num_heads, int block_size, int topk, float softmax_scale, uint16_t* out,
                         float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (q_len < 1 || q_len > kMaxQueryTokens) return MLA_ERR_INVALID_ARG;
  mla_status_t s = check_decode_args(q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table,
                                     max_blocks_per_req, context_lens, topk_idx, batch, num_heads, block_size,
                                     topk, softmax_scale, out, fmt);
  if (s != MLA_OK || batch == 0) return s;
  if (lse && !aligned(lse, 4)) return MLA_ERR_INVALID_ARG;
  const DecodePlan plan = plan_sparse_decode(batch * q_len, num_heads, topk);
  if (plan.workspace > 0) {
    if (workspace_bytes < plan.workspace) return MLA_ERR_WORKSPACE_TOO_SMALL;
    if (!workspace || !aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  }
  return cuda_status(launch_sparse_decode(fmt, q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table,
                                          max_blocks_per_req, context_lens, topk_idx, batch, q_len, num_heads, topk,
                                          softmax_scale, out, lse, workspace, plan, stream));
}

constexpr int kMaxWindow = 0x7FFFFF00;  // a wider window sees everything a 32-bit context can hold

mla_status_t check_dense_args(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                              int64_t kv_block_stride, int64_t num_blocks, const int32_t* block_table,
                              int max_blocks_per_req, const int32_t* context_lens, int batch, int q_len,
                              int num_heads, int block_size, float softmax_scale, int fmt, const uint16_t* out,
                              const float* lse) {
  if (fmt != MLA_KV_NVFP4 && fmt != MLA_KV_FP8) return MLA_ERR_INVALID_ARG;
  if (q_len < 1 || q_len > kMaxQueryTokens) return MLA_ERR_INVALID_ARG;
  // the list pointer's place is taken by the table: these decodes have no list
  mla_status_t s = check_decode_args(q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table,
                                     max_blocks_per_req, context_lens, block_table, batch, num_heads, block_size, 1,
                                     softmax_scale, out, fmt);
  if (s != MLA_OK || batch == 0) return s;
  if (!aligned(q_rope, 16) || (lse && !aligned(lse, 4))) return MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(batch) * q_len * num_heads > 0x7FFFFFFF) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

int64_t window_rows(int q_len, int max_blocks_per_req, int sinks, int window) {
  const int64_t held = static_cast<int64_t>(max_blocks_per_req) * kBlock;
  const int64_t seen = static_cast<int64_t>(sinks) + window + q_len - 1;
  return seen < held ? seen : held;
}
int64_t own_rows(int max_blocks_per_req, int max_context_len) {
  const int64_t held = static_cast<int64_t>(max_blocks_per_req) * kBlock;
  return max_context_len < held ? max_context_len : held;
}
mla_status_t run_dense(int fmt, const DenseArgs& a, const DensePlan& plan, void* workspace, size_t workspace_bytes,
                       cudaStream_t stream) {
  if (plan.workspace > 0) {
    if (workspace_bytes < plan.workspace) return MLA_ERR_WORKSPACE_TOO_SMALL;
    if (!workspace || !aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  }
  return cuda_status(launch_dense_decode(fmt, a, plan, workspace, stream));
}

// Whether two of n x m rows of `dim` elements, row (i, j) at i * s + j * t with
// s, t >= dim, share an element: i s - j t is within dim of 0 for an i in 1..n-1
// and a j in 1..m-1.
bool rows_overlap(int64_t n, int64_t s, int64_t m, int64_t t, int64_t dim) {
  using Wide = __int128;  // strides are the caller's: products may pass 64 bits
  if (n < 2 || m < 2) return false;
  if (static_cast<Wide>(m - 1) * t + dim <= s || static_cast<Wide>(n - 1) * s + dim <= t) return false;  // nested
  if (m > n) return rows_overlap(m, t, n, s, dim);
  for (int64_t j = 1; j < m; ++j) {
    const Wide at = static_cast<Wide>(j) * t, i = at / s;  // the nearest rows of the other kind: i and i + 1
    if ((i >= 1 && i < n && at - i * s < dim) || (i + 1 < n && (i + 1) * s - at < dim)) return true;
  }
  return false;
}
mla_status_t check_heads(const mla_heads_t* h, int64_t n_tokens, int head_dim) {
  if (h->heads < 0) return MLA_ERR_INVALID_ARG;
  if (h->heads == 0 || n_tokens == 0) return MLA_OK;
  if (!h->in || !h->out || !aligned(h->in, 16) || !aligned(h->out, 16)) return MLA_ERR_INVALID_ARG;
  if (h->weight && !aligned(h->weight, 16)) return MLA_ERR_INVALID_ARG;
  // the stride of an axis of one entry is not used
  if (n_tokens > 1 && (h->in_token_stride % 8 || h->out_token_stride % 8)) return MLA_ERR_INVALID_ARG;
  if (h->heads > 1 && (h->in_head_stride % 8 || h->out_head_stride % 8)) return MLA_ERR_INVALID_ARG;
  // no two rows of the output may share an element
  if (n_tokens > 1 && h->out_token_stride < head_dim) return MLA_ERR_INVALID_ARG;
  if (h->heads > 1 && h->out_head_stride < head_dim) return MLA_ERR_INVALID_ARG;
  if (rows_overlap(n_tokens, h->out_token_stride, h->heads, h->out_head_stride, head_dim)) return MLA_ERR_INVALID_ARG;
  if (h->in == h->out && ((n_tokens > 1 && h->in_token_stride != h->out_token_stride) ||
                          (h->heads > 1 && h->in_head_stride != h->out_head_stride)))
    return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}
HeadSet head_set(const mla_heads_t* h) {
  if (h == nullptr || h->heads == 0) return HeadSet{};
  return HeadSet{h->in,           h->out, h->heads, h->in_token_stride, h->in_head_stride, h->out_token_stride,
                 h->out_head_stride, h->weight};
}
mla_status_t check_norm_rope(const mla_heads_t* q, const mla_heads_t* k, int64_t n_tokens, int head_dim,
                             int rope_offset, float eps, const int32_t* positions, const double* inv_freq) {
  if (n_tokens < 0 || !(eps > 0.f) || !std::isfinite(eps)) return MLA_ERR_INVALID_ARG;
  if (q || k) {
    if (head_dim < kRope || head_dim % 8 != 0 || rope_offset < 0 || rope_offset % 8 != 0 ||
        rope_offset > head_dim - kRope)
      return MLA_ERR_INVALID_ARG;
    if (head_dim > 256) return MLA_ERR_UNSUPPORTED;
  }
  for (const mla_heads_t* h : {q, k}) {
    if (h == nullptr) continue;
    const mla_status_t s = check_heads(h, n_tokens, head_dim);
    if (s != MLA_OK) return s;
  }
  if (n_tokens == 0) return MLA_OK;
  if (!positions || !inv_freq || !aligned(positions, 4) || !aligned(inv_freq, 8)) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

constexpr int kMaxNormDim = 16384;
constexpr int64_t kMaxTokens = 0x7FFFFF00;  // of a packed batch: a tile past the last still has a 32-bit number

// Sizes of a packed batch for which every number that the plan and the kernels form fits: of
// the search through the sequences (up to batch + 32), of rows, and of units of work.
bool prompt_sizes_fit(int64_t q_tokens, int64_t kv_tokens, int64_t batch, int64_t num_heads, int64_t num_kv_heads) {
  return q_tokens <= kMaxTokens && kv_tokens <= kMaxTokens && batch <= kMaxTokens &&
         q_tokens * num_heads <= 0x7FFFFFFF && batch * num_kv_heads <= 0x7FFFFFFF;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

namespace {
// Per-device caches of the SM count and the fault word's device address.
// Host threads may drive different devices at once: each device has its own
// slot (an atomic, so the fast path takes no lock), filled once under a
// mutex.  A device index past the table is looked up on every call.
constexpr int kMaxCachedDevices = 64;
std::mutex g_cache_mutex;
std::atomic<int> g_sm_count[kMaxCachedDevices];
std::atomic<unsigned int*> g_fault_word_ptr[kMaxCachedDevices];

int query_sm_count(int dev) {
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) sms = 148;
  return sms;
}
unsigned int* query_fault_word() {
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_fault_word) != cudaSuccess) return nullptr;
  return static_cast<unsigned int*>(p);
}
}  // namespace

int device_sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 0 || dev >= kMaxCachedDevices) return query_sm_count(dev);
  int sms = g_sm_count[dev].load(std::memory_order_acquire);
  if (sms > 0) return sms;
  std::lock_guard<std::mutex> lock(g_cache_mutex);
  sms = g_sm_count[dev].load(std::memory_order_relaxed);
  if (sms <= 0) {
    sms = query_sm_count(dev);
    g_sm_count[dev].store(sms, std::memory_order_release);
  }
  return sms;
}

// The address is cached per device for the life of the process; after a
// cudaDeviceReset the library's device variables may move, so a process that
// resets a device must not call into the library on it again.
unsigned int* fault_word_ptr() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  if (dev < 0 || dev >= kMaxCachedDevices) return query_fault_word();
  unsigned int* p = g_fault_word_ptr[dev].load(std::memory_order_acquire);
  if (p != nullptr) return p;
  std::lock_guard<std::mutex> lock(g_cache_mutex);
  p = g_fault_word_ptr[dev].load(std::memory_order_relaxed);
  if (p == nullptr) {
    p = query_fault_word();
    if (p != nullptr) g_fault_word_ptr[dev].store(p, std::memory_order_release);
  }
  return p;
}

namespace {
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link
// against the driver library); null if unavailable.
EncodeTiledFn encode_tiled() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}
}  // namespace

bool tensor_maps_available() { return encode_tiled() != nullptr; }

cudaError_t set_smem_limit_once(const void* kernel, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (uint64_t{1} << dev) : 0;
  if (bit != 0 && (done->load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit != 0) done->fetch_or(bit, std::memory_order_release);
  return e;
}

bool encode_tensor_map_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t inner,
                          uint64_t rows, uint64_t row_stride, uint32_t box_inner, uint32_t box_rows,
                          CUtensorMapSwizzle swizzle) {
  EncodeTiledFn fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {inner, rows};
  const cuuint64_t strides[1] = {row_stride};
  const cuuint32_t box[2] = {box_inner, box_rows};
  const cuuint32_t estr[2] = {1u, 1u};
  return fn(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_tensor_map_3d(CUtensorMap* map, const void* base, uint64_t inner, uint64_t heads, uint64_t rows,
                          uint64_t head_stride, uint64_t row_stride, uint32_t box_heads, uint32_t box_rows) {
  EncodeTiledFn fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t any = (2 * inner + 15) / 16 * 16;  // for an axis of one entry
  const cuuint64_t dims[3] = {inner, heads, rows};
  const cuuint64_t strides[2] = {heads > 1 ? head_stride : any, rows > 1 ? row_stride : any};
  const cuuint32_t box[3] = {64u, box_heads, box_rows};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_kv_row_bytes(mla_kv_format_t fmt) { return static_cast<size_t>(row_bytes(fmt)); }

const char* mla_status_string(mla_status_t s) {
  switch (s) {
    case MLA_OK: return "MLA_OK";
    case MLA_ERR_INVALID_ARG: return "MLA_ERR_INVALID_ARG";
    case MLA_ERR_UNSUPPORTED: return "MLA_ERR_UNSUPPORTED";
    case MLA_ERR_WORKSPACE_TOO_SMALL: return "MLA_ERR_WORKSPACE_TOO_SMALL";
    case MLA_ERR_CUDA: return "MLA_ERR_CUDA";
  }
  return "MLA_ERR_UNKNOWN";
}

mla_status_t mla_last_cuda_error(int* cuda_err) {
  if (!cuda_err) return MLA_ERR_INVALID_ARG;
  *cuda_err = t_last_cuda_error;
  return MLA_OK;
}

mla_status_t mla_device_fault(unsigned int* word, int clear, mla_stream_t stream) {
  if (!word) return MLA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_fault_word, sizeof(unsigned int), 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && clear) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_fault_word, &zero, sizeof(unsigned int), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  return cuda_status(e);
}

mla_status_t mla_kv_quantize_append(const uint16_t* latent, const uint16_t* rope, const int64_t* slot_mapping,
                                    int64_t n_tokens, void* kv_pool, int64_t num_blocks, int block_size,
                                    int64_t kv_block_stride, mla_kv_format_t fmt, mla_stream_t stream) {
  if (n_tokens < 0 || num_blocks < 0) return MLA_ERR_INVALID_ARG;
  if (fmt != MLA_KV_NVFP4 && fmt != MLA_KV_FP8) return MLA_ERR_INVALID_ARG;
  mla_status_t s = check_block_size(block_size);
  if (s != MLA_OK) return s;
  if (kv_block_stride % 16 != 0 || kv_block_stride < static_cast<int64_t>(block_size) * row_bytes(fmt))
    return MLA_ERR_INVALID_ARG;
  if (n_tokens == 0) return MLA_OK;
  if (!latent || !rope || !slot_mapping || !kv_pool) return MLA_ERR_INVALID_ARG;
  if (!aligned(latent, 16) || !aligned(rope, 4) || !aligned(slot_mapping, 8) || !aligned(kv_pool, 16))
    return MLA_ERR_INVALID_ARG;
  return cuda_status(launch_quantize_append(latent, rope, slot_mapping, n_tokens, kv_pool, num_blocks,
                                            kv_block_stride, fmt, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mla_sparse_decode_workspace_size(int batch, int num_heads, int topk) {
  if (batch <= 0 || num_heads < 16 || num_heads % 16 != 0 || topk < 1) return 0;
  return plan_sparse_decode(batch, num_heads, topk).workspace;
}

mla_status_t mla_sparse_decode_plan(int batch, int num_heads, int topk, int* splits, int* rows_per_split,
                                    int* kernels) {
  if (batch <= 0 || num_heads < 16 || num_heads % 16 != 0 || topk < 1) return MLA_ERR_INVALID_ARG;
  const DecodePlan plan = plan_sparse_decode(batch, num_heads, topk);
  if (splits) *splits = plan.splits;
  if (rows_per_split) *rows_per_split = plan.rows_per_split;
  if (kernels) *kernels = (plan.splits > 1 && !plan.cluster) ? 2 : 1;
  return MLA_OK;
}

mla_status_t mla_sparse_decode_plan_fmt(int fmt, int batch, int num_heads, int topk, int64_t kv_block_stride,
                                        int64_t num_blocks, int* splits, int* rows_per_split, int* kernels,
                                        int* tensor_memory) {
  if (fmt != MLA_KV_NVFP4 && fmt != MLA_KV_FP8) return MLA_ERR_INVALID_ARG;
  if (batch <= 0 || num_heads < 16 || num_heads % 16 != 0 || topk < 1) return MLA_ERR_INVALID_ARG;
  const DecodePlan plan = plan_sparse_decode(batch, num_heads, topk);
  const bool tc = sparse_decode_uses_tc(fmt, num_heads, kv_block_stride, num_blocks);
  int s = plan.splits, rows = plan.rows_per_split, k = (plan.splits > 1 && !plan.cluster) ? 2 : 1;
  if (tc) {
    s = plan_sparse_decode_tc(batch, num_heads, topk, plan.splits);
    rows = (topk + s - 1) / s;
    k = s > 1 ? 2 : 1;
  }
  if (splits) *splits = s;
  if (rows_per_split) *rows_per_split = rows;
  if (kernels) *kernels = k;
  if (tensor_memory) *tensor_memory = tc ? 1 : 0;
  return MLA_OK;
}

mla_status_t mla_sparse_decode(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                               int64_t kv_block_stride, int64_t num_blocks, const int32_t* block_table,
                               int max_blocks_per_req, const int32_t* context_lens, const int32_t* topk_idx,
                               int batch, int num_heads, int block_size, int topk, float softmax_scale,
                               uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                               mla_stream_t stream) {
  return decode_impl(MLA_KV_NVFP4, q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table,
                     max_blocks_per_req, context_lens, topk_idx, batch, 1, num_heads, block_size, topk,
                     softmax_scale, out, lse, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

mla_status_t mla_sparse_decode_fp8(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                                   int64_t kv_block_stride, int64_t num_blocks, const int32_t* block_table,
                                   int max_blocks_per_req, const int32_t* context_lens, const int32_t* topk_idx,
                                   int batch, int num_heads, int block_size, int topk, float softmax_scale,
                                   uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                                   mla_stream_t stream) {
  return decode_impl(MLA_KV_FP8, q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table,
                     max_blocks_per_req, context_lens, topk_idx, batch, 1, num_heads, block_size, topk,
                     softmax_scale, out, lse, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

mla_status_t mla_index_key_quantize_append(const uint16_t* keys, const int64_t* slot_mapping, int64_t n_tokens,
                                           void* idx_key_pool, int64_t num_blocks, int block_size,
                                           int64_t idx_block_stride, mla_stream_t stream) {
  if (n_tokens < 0 || num_blocks < 0) return MLA_ERR_INVALID_ARG;
  mla_status_t s = check_block_size(block_size);
  if (s != MLA_OK) return s;
  if (idx_block_stride % 16 != 0 || idx_block_stride < static_cast<int64_t>(block_size) * (kIdxDim + 4))
    return MLA_ERR_INVALID_ARG;
  if (n_tokens == 0) return MLA_OK;
  if (!keys || !slot_mapping || !idx_key_pool) return MLA_ERR_INVALID_ARG;
  if (!aligned(keys, 16) || !aligned(slot_mapping, 8) || !aligned(idx_key_pool, 16)) return MLA_ERR_INVALID_ARG;
  return cuda_status(launch_index_key_append(keys, slot_mapping, n_tokens, idx_key_pool, num_blocks,
                                             idx_block_stride, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mla_staged_pool_bytes(int batch, int topk) {
  if (batch <= 0 || topk < 1) return 0;
  const int64_t nblk = (topk + kBlock - 1) / kBlock;
  return static_cast<size_t>(batch) * nblk * kBlock * kRowFp8;
}

mla_status_t mla_stage_rows_fp8(const void* kv_pool, int64_t kv_block_stride, int64_t num_blocks,
                                const int32_t* block_table, int max_blocks_per_req, const int32_t* context_lens,
                                const int32_t* topk_idx, int batch, int block_size, int topk, void* staged_pool,
                                int32_t* staged_topk, mla_stream_t stream) {
  if (batch < 0 || topk < 1 || topk > 2048) return MLA_ERR_INVALID_ARG;
  mla_status_t s = check_block_size(block_size);
  if (s != MLA_OK) return s;
  if (batch == 0) return MLA_OK;
  if (!kv_pool || !block_table || !context_lens || !topk_idx || !staged_pool || !staged_topk)
    return MLA_ERR_INVALID_ARG;
  if (!aligned(kv_pool, 16) || !aligned(staged_pool, 16) || !aligned(block_table, 4) ||
      !aligned(context_lens, 4) || !aligned(topk_idx, 4) || !aligned(staged_topk, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_blocks < 0 || max_blocks_per_req < 1) return MLA_ERR_INVALID_ARG;
  if (kv_block_stride % 16 != 0 || kv_block_stride < static_cast<int64_t>(block_size) * kRowNvfp4)
    return MLA_ERR_INVALID_ARG;
  return cuda_status(launch_stage_rows_fp8(kv_pool, kv_block_stride, num_blocks, block_table, max_blocks_per_req,
                                           context_lens, topk_idx, batch, topk, staged_pool, staged_topk, nullptr,
                                           nullptr, reinterpret_cast<cudaStream_t>(stream)));
}

namespace {
// Workspace of the staged decode: staged rows | staged list | identity block
// table | context lengths | the FP8 decode's own split-K workspace.
struct StagedLayout {
  size_t rows, list, table, ctx, decode, total;
};
StagedLayout staged_layout(int batch, int num_heads, int topk) {
  StagedLayout l{};
  const int64_t nblk = (topk + kBlock - 1) / kBlock;
  l.rows = align256(mla_staged_pool_bytes(batch, topk));
  l.list = align256(static_cast<size_t>(batch) * topk * sizeof(int32_t));
  l.table = align256(static_cast<size_t>(batch) * nblk * sizeof(int32_t));
  l.ctx = align256(static_cast<size_t>(batch) * sizeof(int32_t));
  l.decode = align256(plan_sparse_decode(batch, num_heads, topk).workspace);
  l.total = l.rows + l.list + l.table + l.ctx + l.decode;
  return l;
}
}  // namespace

size_t mla_sparse_decode_staged_workspace_size(int batch, int num_heads, int topk) {
  if (batch <= 0 || num_heads < 16 || num_heads % 16 != 0 || topk < 1) return 0;
  return staged_layout(batch, num_heads, topk).total;
}

mla_status_t mla_sparse_decode_staged(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                                      int64_t kv_block_stride, int64_t num_blocks, const int32_t* block_table,
                                      int max_blocks_per_req, const int32_t* context_lens, const int32_t* topk_idx,
                                      int batch, int num_heads, int block_size, int topk, float softmax_scale,
                                      uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                                      mla_stream_t stream) {
  mla_status_t s = check_decode_args(q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table,
                                     max_blocks_per_req, context_lens, topk_idx, batch, num_heads, block_size, topk,
                                     softmax_scale, out, MLA_KV_NVFP4);
  if (s != MLA_OK || batch == 0) return s;
  if (lse && !aligned(lse, 4)) return MLA_ERR_INVALID_ARG;
  const StagedLayout l = staged_layout(batch, num_heads, topk);
  if (workspace_bytes < l.total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (!workspace || !aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* rows = ws;
  int32_t* list = reinterpret_cast<int32_t*>(ws + l.rows);
  int32_t* table = reinterpret_cast<int32_t*>(ws + l.rows + l.list);
  int32_t* ctx = reinterpret_cast<int32_t*>(ws + l.rows + l.list + l.table);
  void* dec_ws = ws + l.rows + l.list + l.table + l.ctx;
  const int nblk = (topk + kBlock - 1) / kBlock;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_stage_rows_fp8(kv_pool, kv_block_stride, num_blocks, block_table, max_blocks_per_req,
                                        context_lens, topk_idx, batch, topk, rows, list, table, ctx, st);
  if (e != cudaSuccess) return cuda_status(e);
  const DecodePlan plan = plan_sparse_decode(batch, num_heads, topk);
  return cuda_status(launch_sparse_decode(MLA_KV_FP8, q_nope, q_rope, rows, static_cast<int64_t>(kBlock) * kRowFp8,
                                          static_cast<int64_t>(batch) * nblk, table, nblk, ctx, list, batch, 1,
                                          num_heads, topk, softmax_scale, out, lse, dec_ws, plan, st));
}

size_t mla_sparse_decode_mtp_workspace_size(int batch, int q_len, int num_heads, int topk) {
  if (batch <= 0 || q_len < 1 || q_len > kMaxQueryTokens || num_heads < 16 || num_heads % 16 != 0 || topk < 1)
    return 0;
  return plan_sparse_decode(batch * q_len, num_heads, topk).workspace;
}

mla_status_t mla_sparse_decode_mtp(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                                   int64_t kv_block_stride, int64_t num_blocks, const int32_t* block_table,
                                   int max_blocks_per_req, const int32_t* context_lens, const int32_t* topk_idx,
                                   int batch, int q_len, int num_heads, int block_size, int topk, float softmax_scale,
                                   mla_kv_format_t fmt, uint16_t* out, float* lse, void* workspace,
                                   size_t workspace_bytes, mla_stream_t stream) {
  if (fmt != MLA_KV_NVFP4 && fmt != MLA_KV_FP8) return MLA_ERR_INVALID_ARG;
  return decode_impl(fmt, q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table, max_blocks_per_req,
                     context_lens, topk_idx, batch, q_len, num_heads, block_size, topk, softmax_scale, out, lse,
                     workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

size_t mla_topk_workspace_size(int batch, int max_context_len, int topk) {
  if (batch <= 0 || max_context_len < 0 || topk < 1) return 0;
  return topk_workspace_bytes(batch, max_context_len, topk);
}

mla_status_t mla_topk(const float* scores, int64_t score_row_stride, const int32_t* context_lens, int batch,
                      int topk, int max_context_len, int32_t* topk_out, void* workspace, size_t workspace_bytes,
                      mla_stream_t stream) {
  if (batch < 0 || topk < 1 || topk > 2048 || max_context_len < 0) return MLA_ERR_INVALID_ARG;
  if (batch == 0) return MLA_OK;
  if (!scores || !context_lens || !topk_out) return MLA_ERR_INVALID_ARG;
  if (score_row_stride < max_context_len || !aligned(scores, 4) || !aligned(topk_out, 4)) return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < topk_workspace_bytes(batch, max_context_len, topk)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (!workspace || !aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  return cuda_status(launch_topk(scores, score_row_stride, context_lens, batch, topk, max_context_len, topk_out,
                                 workspace, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mla_indexer_topk_workspace_size(int batch, int max_context_len, int topk) {
  if (batch <= 0 || max_context_len <= 0 || topk < 1) return 0;
  const size_t scores = align256(static_cast<size_t>(batch) * max_context_len * sizeof(float));
  return scores + align256(topk_workspace_bytes(batch, max_context_len, topk));
}

mla_status_t mla_indexer_topk(const uint16_t* q_idx, const float* head_w, const void* idx_key_pool,
                              int64_t idx_block_stride, int64_t num_blocks, const int32_t* block_table,
                              int max_blocks_per_req, const int32_t* context_lens, int batch, int n_idx_heads,
                              int block_size, int topk, int32_t* topk_out, float* scores_out, int max_context_len,
                              void* workspace, size_t workspace_bytes, mla_stream_t stream) {
  if (batch < 0 || topk < 1 || topk > 2048 || max_context_len < 0) return MLA_ERR_INVALID_ARG;
  mla_status_t s = check_block_size(block_size);
  if (s != MLA_OK) return s;
  if (n_idx_heads != 8 && n_idx_heads != 16 && n_idx_heads != 32 && n_idx_heads != 64) {
    return (n_idx_heads > 0 && n_idx_heads % 8 == 0 && n_idx_heads <= 64) ? MLA_ERR_UNSUPPORTED
                                                                          : MLA_ERR_INVALID_ARG;
  }
  if (batch == 0) return MLA_OK;
  if (!q_idx || !head_w || !idx_key_pool || !block_table || !context_lens || !topk_out) return MLA_ERR_INVALID_ARG;
  if (!aligned(q_idx, 16) || !aligned(head_w, 4) || !aligned(idx_key_pool, 16)) return MLA_ERR_INVALID_ARG;
  if (idx_block_stride % 16 != 0 || idx_block_stride < static_cast<int64_t>(block_size) * (kIdxDim + 4))
    return MLA_ERR_INVALID_ARG;
  if (num_blocks < 0 || max_blocks_per_req < 1) return MLA_ERR_INVALID_ARG;
  const size_t need = mla_indexer_topk_workspace_size(batch, max_context_len, topk);
  float* scores = scores_out;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (need > 0) {
    if (workspace_bytes < need) return MLA_ERR_WORKSPACE_TOO_SMALL;
    if (!workspace || !aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  }
  if (scores == nullptr) scores = reinterpret_cast<float*>(ws);
  else if (!aligned(scores, 4)) return MLA_ERR_INVALID_ARG;
  const size_t scores_bytes = align256(static_cast<size_t>(batch) * max_context_len * sizeof(float));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_indexer_scores(q_idx, head_w, idx_key_pool, idx_block_stride, num_blocks, block_table,
                                        max_blocks_per_req, context_lens, batch, n_idx_heads, max_context_len, scores,
                                        max_context_len, st);
  if (e != cudaSuccess) return cuda_status(e);
  return cuda_status(launch_topk(scores, max_context_len, context_lens, batch, topk, max_context_len, topk_out,
                                 ws ? ws + scores_bytes : nullptr, st));
}

mla_status_t mla_block_table_extend(const int32_t* context_lens, const int32_t* new_lens, int batch,
                                    int32_t* block_table, int max_blocks_per_req, const int32_t* free_blocks,
                                    int64_t free_capacity, const int64_t* free_state, int64_t num_blocks,
                                    int block_size, int64_t* slot_mapping, int32_t* positions, int64_t num_slots,
                                    int32_t* query_start, int32_t* context_lens_out, int64_t* free_state_out,
                                    mla_stream_t stream) {
  if (batch < 0 || max_blocks_per_req < 1 || free_capacity < 0 || num_blocks < 0 || num_slots < 0)
    return MLA_ERR_INVALID_ARG;
  mla_status_t s = check_block_size(block_size);
  if (s != MLA_OK) return s;
  if (num_slots > 0x7FFFFFFF) return MLA_ERR_INVALID_ARG;  // starts are 32-bit
  if (batch > 0 && (!context_lens || !new_lens || !block_table || !context_lens_out)) return MLA_ERR_INVALID_ARG;
  if (num_slots > 0 && (!slot_mapping || !positions)) return MLA_ERR_INVALID_ARG;
  if (!free_state || !free_state_out || !query_start || (free_capacity > 0 && !free_blocks))
    return MLA_ERR_INVALID_ARG;
  if (!aligned(context_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) || !aligned(free_blocks, 4) ||
      !aligned(free_state, 8) || !aligned(slot_mapping, 8) || !aligned(positions, 4) || !aligned(query_start, 4) ||
      !aligned(context_lens_out, 4) || !aligned(free_state_out, 8))
    return MLA_ERR_INVALID_ARG;
  const ExtendArgs a{context_lens,  new_lens,   batch,        block_table, max_blocks_per_req,
                     free_blocks,   free_capacity, free_state, num_blocks,  slot_mapping,
                     positions,     num_slots,  query_start,  context_lens_out, free_state_out};
  return cuda_status(launch_block_table_extend(a, reinterpret_cast<cudaStream_t>(stream)));
}

mla_status_t mla_qk_norm_rope(const mla_heads_t* q, const mla_heads_t* k, int64_t n_tokens, int head_dim,
                              int rope_offset, int interleaved, float eps, const int32_t* positions,
                              const double* inv_freq, mla_stream_t stream) {
  if (!q && !k) return MLA_ERR_INVALID_ARG;
  mla_status_t s = check_norm_rope(q, k, n_tokens, head_dim, rope_offset, eps, positions, inv_freq);
  if (s != MLA_OK || n_tokens == 0) return s;
  NormRopeArgs a{};
  a.set[0] = head_set(q);
  a.set[1] = head_set(k);
  a.tokens = n_tokens;
  a.dim = head_dim;
  a.rope_offset = rope_offset;
  a.eps = eps;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.interleaved = interleaved != 0;
  return cuda_status(launch_norm_rope(a, reinterpret_cast<cudaStream_t>(stream)));
}

mla_status_t mla_kv_norm_rope_append(const uint16_t* kv, int64_t kv_token_stride, const uint16_t* latent_weight,
                                     const mla_heads_t* q, int head_dim, int rope_offset, int interleaved, float eps,
                                     const int32_t* positions, const double* inv_freq, const int64_t* slot_mapping,
                                     int64_t n_tokens, void* kv_pool, int64_t num_blocks, int block_size,
                                     int64_t kv_block_stride, mla_kv_format_t fmt, mla_stream_t stream) {
  if (num_blocks < 0 || (fmt != MLA_KV_NVFP4 && fmt != MLA_KV_FP8)) return MLA_ERR_INVALID_ARG;
  mla_status_t s = check_block_size(block_size);
  if (s != MLA_OK) return s;
  if (kv_block_stride % 16 != 0 || kv_block_stride < static_cast<int64_t>(block_size) * row_bytes(fmt))
    return MLA_ERR_INVALID_ARG;
  s = check_norm_rope(q, nullptr, n_tokens, head_dim, rope_offset, eps, positions, inv_freq);
  if (s != MLA_OK || n_tokens == 0) return s;
  if (!kv || !latent_weight || !slot_mapping || !kv_pool) return MLA_ERR_INVALID_ARG;
  if (!aligned(kv, 16) || !aligned(latent_weight, 16) || !aligned(slot_mapping, 8) || !aligned(kv_pool, 16) ||
      (n_tokens > 1 && kv_token_stride % 8 != 0))
    return MLA_ERR_INVALID_ARG;
  NormRopeArgs a{};
  a.set[0] = head_set(q);
  a.tokens = n_tokens;
  a.dim = q ? head_dim : kRope;
  a.rope_offset = rope_offset;
  a.eps = eps;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.interleaved = interleaved != 0;
  a.kv = kv;
  a.kv_token = kv_token_stride;
  a.latent_weight = latent_weight;
  a.slot_mapping = slot_mapping;
  a.pool = static_cast<uint8_t*>(kv_pool);
  a.num_blocks = num_blocks;
  a.block_stride = kv_block_stride;
  a.fmt = fmt;
  return cuda_status(launch_norm_rope(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mla_window_decode_workspace_size(int batch, int q_len, int num_heads, int max_blocks_per_req, int sinks,
                                        int window) {
  if (batch <= 0 || q_len < 1 || num_heads < 16 || num_heads % 16 != 0 || max_blocks_per_req < 1 || sinks < 0 ||
      window < 1)
    return 0;
  return plan_dense_decode(batch, q_len, num_heads, window_rows(q_len, max_blocks_per_req, sinks, window), 0).workspace;
}

mla_status_t mla_window_decode(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                               int64_t kv_block_stride, int64_t num_blocks, const int32_t* block_table,
                               int max_blocks_per_req, const int32_t* context_lens, int batch, int q_len,
                               int num_heads, int block_size, int sinks, int window, float softmax_scale,
                               mla_kv_format_t fmt, uint16_t* out, float* lse, void* workspace,
                               size_t workspace_bytes, mla_stream_t stream) {
  if (sinks < 0 || window < 1) return MLA_ERR_INVALID_ARG;
  mla_status_t s = check_dense_args(q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table,
                                    max_blocks_per_req, context_lens, batch, q_len, num_heads, block_size,
                                    softmax_scale, fmt, out, lse);
  if (s != MLA_OK || batch == 0) return s;
  DenseArgs a{};
  a.q_nope = q_nope;
  a.q_rope = q_rope;
  a.pool = static_cast<const uint8_t*>(kv_pool);
  a.block_stride = kv_block_stride;
  a.num_blocks = num_blocks;
  a.block_table = block_table;
  a.max_blocks = max_blocks_per_req;
  a.ctx_lens = context_lens;
  a.max_context = 0x7FFFFFFF;
  a.batch = batch;
  a.q_len = q_len;
  a.num_heads = num_heads;
  a.sinks = sinks;
  a.window = window < kMaxWindow ? window : kMaxWindow;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.out = out;
  a.lse = lse;
  const DensePlan plan =
      plan_dense_decode(batch, q_len, num_heads, window_rows(q_len, max_blocks_per_req, sinks, window), 0);
  return run_dense(fmt, a, plan, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

size_t mla_prefix_decode_workspace_size(int batch, int q_len, int num_heads, int prefix_len, int max_blocks_per_req,
                                        int max_context_len) {
  if (batch <= 0 || q_len < 1 || num_heads < 16 || num_heads % 16 != 0 || prefix_len < 0 || max_blocks_per_req < 1 ||
      max_context_len < 0)
    return 0;
  return plan_dense_decode(batch, q_len, num_heads, own_rows(max_blocks_per_req, max_context_len), prefix_len).workspace;
}

mla_status_t mla_prefix_decode(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                               int64_t kv_block_stride, int64_t num_blocks, const int32_t* prefix_table,
                               int prefix_len, const int32_t* block_table, int max_blocks_per_req,
                               const int32_t* context_lens, int batch, int q_len, int num_heads, int block_size,
                               int max_context_len, float softmax_scale, mla_kv_format_t fmt, uint16_t* out,
                               float* lse, void* workspace, size_t workspace_bytes, mla_stream_t stream) {
  if (prefix_len < 0 || prefix_len > kMaxWindow || max_context_len < 0) return MLA_ERR_INVALID_ARG;
  mla_status_t s = check_dense_args(q_nope, q_rope, kv_pool, kv_block_stride, num_blocks, block_table,
                                    max_blocks_per_req, context_lens, batch, q_len, num_heads, block_size,
                                    softmax_scale, fmt, out, lse);
  if (s != MLA_OK || batch == 0) return s;
  if (prefix_len > 0 && (!prefix_table || !aligned(prefix_table, 4))) return MLA_ERR_INVALID_ARG;
  DenseArgs a{};
  a.q_nope = q_nope;
  a.q_rope = q_rope;
  a.pool = static_cast<const uint8_t*>(kv_pool);
  a.block_stride = kv_block_stride;
  a.num_blocks = num_blocks;
  a.prefix_table = prefix_table;
  a.prefix_len = prefix_len;
  a.block_table = block_table;
  a.max_blocks = max_blocks_per_req;
  a.ctx_lens = context_lens;
  a.max_context = max_context_len;
  a.batch = batch;
  a.q_len = q_len;
  a.num_heads = num_heads;
  a.sinks = 0;
  a.window = kMaxWindow;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.out = out;
  a.lse = lse;
  const DensePlan plan =
      plan_dense_decode(batch, q_len, num_heads, own_rows(max_blocks_per_req, max_context_len), prefix_len);
  return run_dense(fmt, a, plan, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

mla_status_t mla_add_norm_quant(const uint16_t* x, int64_t x_stride, mla_residual_t residual_type,
                                const void* residual, int64_t residual_stride, void* residual_out,
                                int64_t residual_out_stride, const uint16_t* weight, int64_t n_tokens, int dim,
                                int group, float eps, uint8_t* codes, float* scales, mla_stream_t stream) {
  if (n_tokens < 0 || dim < 8 || dim % 8 != 0 || !(eps > 0.f) || !std::isfinite(eps)) return MLA_ERR_INVALID_ARG;
  if (residual_type != MLA_RESIDUAL_NONE && residual_type != MLA_RESIDUAL_BF16 && residual_type != MLA_RESIDUAL_F32)
    return MLA_ERR_INVALID_ARG;
  if (group < 0 || group % 8 != 0) return MLA_ERR_INVALID_ARG;
  if ((group != 0 && group != 128) || dim > kMaxNormDim) return MLA_ERR_UNSUPPORTED;
  if (n_tokens == 0) return MLA_OK;
  if (!x || !weight || !codes || !scales) return MLA_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(codes, 8) || !aligned(scales, 4)) return MLA_ERR_INVALID_ARG;
  if (n_tokens > 1 && x_stride % 8 != 0) return MLA_ERR_INVALID_ARG;
  if (residual_type != MLA_RESIDUAL_NONE) {
    if (!residual || !residual_out || !aligned(residual, 16) || !aligned(residual_out, 16)) return MLA_ERR_INVALID_ARG;
    const int unit = residual_type == MLA_RESIDUAL_BF16 ? 8 : 4;  // 16 bytes
    if (n_tokens > 1 && (residual_stride % unit != 0 || residual_out_stride % unit != 0 || residual_out_stride < dim ||
                         (residual == residual_out && residual_stride != residual_out_stride)))
      return MLA_ERR_INVALID_ARG;
  }
  AddNormArgs a{};
  a.x = x;
  a.x_stride = x_stride;
  a.residual_type = residual_type;
  a.residual = residual;
  a.res_stride = residual_stride;
  a.residual_out = residual_out;
  a.res_out_stride = residual_out_stride;
  a.weight = weight;
  a.tokens = n_tokens;
  a.dim = dim;
  a.group = group;
  a.scale_groups = group == 0 ? 1 : (dim + group - 1) / group;
  a.eps = eps;
  a.inv_dim = 1.f / static_cast<float>(dim);
  a.codes = codes;
  a.scales = scales;
  return cuda_status(launch_add_norm_quant(a, reinterpret_cast<cudaStream_t>(stream)));
}

mla_status_t mla_fp4_matvec(const void* x, mla_x_type_t x_type, int64_t x_token_stride, int64_t x_group_stride,
                            const float* x_scales, int x_scale_groups, const uint8_t* codes, const uint8_t* scales,
                            const float* weight_scale, int64_t n_tokens, int groups, int n, int k, void* out,
                            mla_out_type_t out_type, int64_t out_token_stride, int64_t out_group_stride,
                            mla_stream_t stream) {
  if (n_tokens < 0 || groups < 0 || n < 0 || k < 16 || k % 16 != 0) return MLA_ERR_INVALID_ARG;
  if ((x_type != MLA_X_BF16 && x_type != MLA_X_E4M3) || (out_type != MLA_OUT_BF16 && out_type != MLA_OUT_F32))
    return MLA_ERR_INVALID_ARG;
  const int pieces = (k - 1) / 128 + 1;
  if (x_type == MLA_X_E4M3 && x_scale_groups != 1 && x_scale_groups != pieces) return MLA_ERR_INVALID_ARG;
  if (k % 32 != 0 || groups > 65535 || n_tokens > 32 * 65535) return MLA_ERR_UNSUPPORTED;
  if (n_tokens == 0 || groups == 0 || n == 0) return MLA_OK;
  if (!x || !codes || !scales || !out) return MLA_ERR_INVALID_ARG;
  const int unit = x_type == MLA_X_BF16 ? 8 : 16;  // 16 bytes
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 2) || !aligned(weight_scale, 4) ||
      !aligned(out, out_type == MLA_OUT_BF16 ? 2 : 4))
    return MLA_ERR_INVALID_ARG;
  if ((n_tokens > 1 && x_token_stride % unit != 0) || (groups > 1 && x_group_stride % unit != 0))
    return MLA_ERR_INVALID_ARG;
  if (x_type == MLA_X_E4M3 && (!x_scales || !aligned(x_scales, 4))) return MLA_ERR_INVALID_ARG;
  // no two rows of the output may share an element
  if ((n_tokens > 1 && out_token_stride < n) || (groups > 1 && out_group_stride < n) ||
      rows_overlap(n_tokens, out_token_stride, groups, out_group_stride, n))
    return MLA_ERR_INVALID_ARG;
  MatvecArgs a{};
  a.x = x;
  a.x_codes = x_type == MLA_X_E4M3;
  a.x_token = x_token_stride;
  a.x_group = x_group_stride;
  a.x_scales = x_scales;
  a.x_scale_groups = x_scale_groups;
  a.codes = codes;
  a.scales = scales;
  a.weight_scale = weight_scale;
  a.tokens = n_tokens;
  a.groups = groups;
  a.n = n;
  a.k = k;
  a.out = out;
  a.out_float = out_type == MLA_OUT_F32;
  a.out_token = out_token_stride;
  a.out_group = out_group_stride;
  return cuda_status(launch_fp4_matvec(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mla_prompt_attention_workspace_size(int64_t q_tokens, int64_t kv_tokens, int batch, int num_heads,
                                           int num_kv_heads, int v_dim) {
  if (q_tokens <= 0 || kv_tokens < 0 || batch <= 0 || num_kv_heads < 1 || num_heads < 1 ||
      num_heads % num_kv_heads != 0 || num_heads / num_kv_heads > 128 || v_dim < 8 ||
      !prompt_sizes_fit(q_tokens, kv_tokens, batch, num_heads, num_kv_heads))
    return 0;
  return plan_prompt_attention(q_tokens, kv_tokens, batch, num_heads, num_kv_heads, v_dim).workspace;
}

mla_status_t mla_prompt_attention_plan(int64_t q_tokens, int64_t kv_tokens, int batch, int num_heads, int num_kv_heads,
                                       int v_dim, int* row_tiles, int* slices, int64_t* units, int* variant) {
  if (q_tokens <= 0 || kv_tokens < 0 || batch <= 0 || num_kv_heads < 1 || num_heads < 1 ||
      num_heads % num_kv_heads != 0 || v_dim < 8 || v_dim % 8 != 0)
    return MLA_ERR_INVALID_ARG;
  if (v_dim > 128 || num_heads / num_kv_heads > 128 ||
      !prompt_sizes_fit(q_tokens, kv_tokens, batch, num_heads, num_kv_heads))
    return MLA_ERR_UNSUPPORTED;
  const PromptPlan plan = plan_prompt_attention(q_tokens, kv_tokens, batch, num_heads, num_kv_heads, v_dim);
  if (row_tiles) *row_tiles = plan.unit_tiles;
  if (slices) *slices = plan.splits;
  if (units) *units = plan.places * num_kv_heads * plan.splits;
  if (variant) *variant = plan.variant;
  return MLA_OK;
}

mla_status_t mla_prompt_attention(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, const uint16_t* k,
                                  int64_t k_token_stride, int64_t k_head_stride, const uint16_t* v,
                                  int64_t v_token_stride, int64_t v_head_stride, const int32_t* query_start,
                                  const int32_t* kv_start, int batch, int64_t q_tokens, int64_t kv_tokens,
                                  int num_heads, int num_kv_heads, int qk_dim, int v_dim, int causal,
                                  float softmax_scale, uint16_t* out, int64_t out_token_stride,
                                  int64_t out_head_stride, float* lse, void* workspace, size_t workspace_bytes,
                                  mla_stream_t stream) {
  if (batch < 0 || q_tokens < 0 || kv_tokens < 0 || num_heads < 1 || num_kv_heads < 1 ||
      num_heads % num_kv_heads != 0 || qk_dim < 8 || qk_dim % 8 != 0 || v_dim < 8 || v_dim % 8 != 0 ||
      !std::isfinite(softmax_scale))
    return MLA_ERR_INVALID_ARG;
  if (qk_dim > 192 || v_dim > 128 || num_heads / num_kv_heads > 128 || q_tokens > kMaxTokens || kv_tokens > kMaxTokens)
    return MLA_ERR_UNSUPPORTED;
  if (batch == 0 || q_tokens == 0) return MLA_OK;
  if (!prompt_sizes_fit(q_tokens, kv_tokens, batch, num_heads, num_kv_heads)) return MLA_ERR_UNSUPPORTED;
  if (!q || !query_start || !kv_start || !out || (kv_tokens > 0 && (!k || !v))) return MLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(query_start, 4) ||
      !aligned(kv_start, 4) || !aligned(lse, 4))
    return MLA_ERR_INVALID_ARG;
  // the stride of an axis of one entry is not used
  if ((q_tokens > 1 && (q_token_stride % 8 || out_token_stride % 8)) ||
      (num_heads > 1 && (q_head_stride % 8 || out_head_stride % 8)) ||
      (kv_tokens > 1 && (k_token_stride % 8 || v_token_stride % 8)) ||
      (kv_tokens > 0 && num_kv_heads > 1 && (k_head_stride % 8 || v_head_stride % 8)))
    return MLA_ERR_INVALID_ARG;
  // rows that overlap, and so an axis repeated by a stride of 0, are nothing the copy engine's
  // descriptions promise
  if ((q_tokens > 1 && q_token_stride < qk_dim) || (num_heads > 1 && q_head_stride < qk_dim) ||
      (kv_tokens > 1 && (k_token_stride < qk_dim || v_token_stride < v_dim)) ||
      (kv_tokens > 0 && num_kv_heads > 1 && (k_head_stride < qk_dim || v_head_stride < v_dim)))
    return MLA_ERR_UNSUPPORTED;
  if ((q_tokens > 1 && out_token_stride < v_dim) || (num_heads > 1 && out_head_stride < v_dim) ||
      rows_overlap(q_tokens, out_token_stride, num_heads, out_head_stride, v_dim))
    return MLA_ERR_INVALID_ARG;
  const PromptPlan plan = plan_prompt_attention(q_tokens, kv_tokens, batch, num_heads, num_kv_heads, v_dim);
  if (plan.places * num_kv_heads * plan.splits > 0x7FFFFFFF) return MLA_ERR_UNSUPPORTED;
  if (plan.workspace > 0) {
    if (workspace_bytes < plan.workspace) return MLA_ERR_WORKSPACE_TOO_SMALL;
    if (!workspace || !aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  }
  PromptArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.k_token = k_token_stride;
  a.k_head = k_head_stride;
  a.v_token = v_token_stride;
  a.v_head = v_head_stride;
  a.q_tokens = static_cast<int>(q_tokens);
  a.kv_tokens = static_cast<int>(kv_tokens);
  a.batch = batch;
  a.q_start = query_start;
  a.kv_start = kv_start;
  a.heads = num_heads;
  a.kv_heads = num_kv_heads;
  a.dk = qk_dim;
  a.dv = v_dim;
  a.causal = causal != 0;
  a.negate = softmax_scale < 0.f;
  // a scale of 0 makes all weights equal, but must keep what is masked at -infinity
  // (and one past float's range, finite: a score of 0 stays 0)
  a.scale_log2 = std::fmin(std::fmax(std::fabs(softmax_scale) * 1.4426950408889634f, 1.401298464324817e-45f), 3.402823466e38f);
  a.out = out;
  a.out_token = out_token_stride;
  a.out_head = out_head_stride;
  a.lse = lse;
  bool described = false;
  const cudaError_t e =
      launch_prompt_attention(a, plan, workspace, reinterpret_cast<cudaStream_t>(stream), &described);
  return described ? cuda_status(e) : MLA_ERR_UNSUPPORTED;
}

}  // extern "C"
