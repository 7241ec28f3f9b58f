/*
 * mla_nvfp4.h -- C ABI of libmla_nvfp4.so: sparse multi-head latent attention
 * (MLA) decode over a paged latent KV cache stored as NVFP4 (352-byte rows)
 * or FP8 (576-byte rows), for NVIDIA GB300 (sm_103a).
 *
 * What the operations are, and where they are defined:
 *
 *  - The cached row.  A token's cache entry is a 512-value latent and a
 *    64-value rotary key shared by all heads (no head axis); every attention head reads the
 *    same row ("Prime Inference: serving GLM-5.3 to agents is a KV-cache
 *    problem", section "Prefill topology").  Stored as NVFP4 it is 256 bytes
 *    of 4-bit e2m1 codes, 32 one-byte e4m3 scales (one per 16 latent values)
 *    and 64 one-byte e4m3 rope values = 352 bytes; stored as FP8 it is 512 +
 *    64 e4m3 bytes = 576 bytes (same page, section "Four bits per latent
 *    value: where 352 comes from", row table).
 *  - Sparse selection.  The indexer rates all preceding tokens and attention
 *    reads at most top-k = 2,048 of them ("GLM-5.3 PCP/DCP long-context on
 *    H200", section 1; "Prime Inference", section "Decode: TP4, and the
 *    copies it keeps", index_topk 2048).  An indexer key is 128 e4m3 bytes
 *    and a float scale (PCP/DCP page, section 3).
 *  - Decode.  The selected rows are gathered through the block table,
 *    unpacked on chip, scored against every head's absorbed query, soft-maxed
 *    and blended, with no FP8 or BF16 copy written to memory ("Prime
 *    Inference", section "A kernel that reads four bits directly", figure
 *    "staged vs native decode"); when a context is shorter than top-k the
 *    list carries -1 entries, which are skipped (same section).
 *
 * Row layout inside the 352 bytes (the pages give only the totals):
 *   [0,256)   latent codes, element 2i in the low nibble of byte i
 *   [256,288) e4m3 scale g for latent elements [16g, 16g+16)
 *   [288,352) rope, e4m3
 * FP8 row: [0,512) latent e4m3, [512,576) rope e4m3.
 * Quantization: S_g = e4m3_rn_satfinite(max_i |x_i| / 6) (IEEE float32
 * division), code_i = e2m1_rn_satfinite(x_i / S_g), ties to even, the sign
 * bit copies the sign of x_i; a group whose S_g encodes to 0 stores sixteen
 * 0x0 codes; rope and FP8 latent values are e4m3_rn_satfinite(x).
 *
 * Conventions for every entry point:
 *  - All pointers marked "device" are CUDA device pointers on the current
 *    device; the caller owns every buffer.  The library allocates nothing and
 *    keeps no per-call state; scratch memory comes in through `workspace`.
 *  - Work is enqueued on `stream` and returns immediately (asynchronous).
 *  - Host-side argument errors return MLA_ERR_INVALID_ARG or
 *    MLA_ERR_UNSUPPORTED synchronously, before any launch; a launch failure
 *    returns MLA_ERR_CUDA and mla_last_cuda_error() gives the CUDA code.
 *  - Device data is never trusted: a top-k entry outside [0, context_len)
 *    (including -1), a logical block past max_blocks_per_req and a physical
 *    block id outside [0, num_blocks) are skipped (no load, no weight), and
 *    an out-of-range slot in mla_kv_quantize_append is not written.
 *  - bf16 arguments are passed as uint16_t bit patterns.
 *  - Every bounded device wait that runs out sets a bit in a library-wide
 *    device fault word (see mla_device_fault) instead of hanging; it never
 *    traps.
 */
#ifndef MLA_NVFP4_H
#define MLA_NVFP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* mla_stream_t; /* the same type as cudaStream_t */

typedef enum {
  MLA_OK = 0,
  MLA_ERR_INVALID_ARG = 1,        /* null pointer, bad size, misalignment */
  MLA_ERR_UNSUPPORTED = 2,        /* a valid value this build does not handle */
  MLA_ERR_WORKSPACE_TOO_SMALL = 3,
  MLA_ERR_CUDA = 4                /* a CUDA call or launch failed */
} mla_status_t;

typedef enum {
  MLA_KV_NVFP4 = 0, /* 352-byte rows */
  MLA_KV_FP8 = 1    /* 576-byte rows */
} mla_kv_format_t;

/* Bytes of one cached row: 352 (NVFP4), 576 (FP8), 0 for an unknown format. */
size_t mla_kv_row_bytes(mla_kv_format_t fmt);

/* A static, human-readable name of a status code. */
const char* mla_status_string(mla_status_t s);

/* The CUDA error code behind this thread's last MLA_ERR_CUDA (0 if none).
 * Thread-local; returns MLA_ERR_INVALID_ARG if cuda_err is NULL. */
mla_status_t mla_last_cuda_error(int* cuda_err);

/* Reads (and, if `clear` is nonzero, resets) the device fault word of the
 * current device: bit 0 = a decode wait ran out, bit 1 = an indexer or top-k
 * wait ran out, bit 2 = a wait of the prompt attention ran out.  Synchronises
 * `stream`.  A nonzero word means some output of an earlier call is incomplete. */
mla_status_t mla_device_fault(unsigned int* word, int clear, mla_stream_t stream);

/*
 * Quantize-on-write ("Prime Inference", section "Four bits per latent
 * value"; Prime Intellect's post: NVFP4 is the storage format).
 *
 *   latent        device bf16 [n_tokens, 512], row stride 512
 *   rope          device bf16 [n_tokens, 64], row stride 64
 *   slot_mapping  device int64 [n_tokens]; token n is written to block
 *                 slot / block_size, row slot % block_size; a negative slot
 *                 or one at or past num_blocks * block_size is skipped
 *   kv_pool       device, 16-byte aligned; block b starts at
 *                 kv_pool + b * kv_block_stride
 *   kv_block_stride  bytes, a multiple of 16, >= block_size * row bytes
 *   block_size    64 (other powers of two: MLA_ERR_UNSUPPORTED)
 * n_tokens == 0 is a no-op.  Two tokens with the same slot race.
 */
mla_status_t mla_kv_quantize_append(const uint16_t* latent, const uint16_t* rope, const int64_t* slot_mapping,
                                    int64_t n_tokens, void* kv_pool, int64_t num_blocks, int block_size,
                                    int64_t kv_block_stride, mla_kv_format_t fmt, mla_stream_t stream);

/*
 * Quantize-on-write of the indexer's keys ("GLM-5.3 PCP/DCP long-context on
 * H200", section 3: a key is 128 e4m3 bytes and a float scale).  Per
 * token: s = max_d |k_d| / 448 and code_d = e4m3_rn_satfinite(k_d / s), both
 * divisions IEEE float32; a key whose values are all zero stores s = 0 and
 * 128 zero codes.  Block layout (the layout mla_indexer_topk reads): block b
 * at idx_key_pool + b * idx_block_stride holds block_size x 128 code bytes,
 * then block_size float scales.
 *
 *   keys          device bf16 [n_tokens, 128], 16-byte aligned
 *   slot_mapping  device int64 [n_tokens]; as for mla_kv_quantize_append
 *                 (a negative or out-of-pool slot is skipped)
 *   idx_key_pool  device, 16-byte aligned
 *   idx_block_stride  bytes, a multiple of 16, >= block_size * 132
 *   block_size    64
 * n_tokens == 0 is a no-op.  Two tokens with the same slot race.
 */
mla_status_t mla_index_key_quantize_append(const uint16_t* keys, const int64_t* slot_mapping, int64_t n_tokens,
                                           void* idx_key_pool, int64_t num_blocks, int block_size,
                                           int64_t idx_block_stride, mla_stream_t stream);

/*
 * Absorbed-form sparse MLA decode over the NVFP4 cache ("Prime Inference",
 * section "A kernel that reads four bits directly").  For request b and head
 * h, with V_b = { t in topk_idx[b, :] : 0 <= t < context_lens[b] } (counted
 * with multiplicity) and c_t, r_t the dequantized latent and rope of token t
 * (logical block t / 64 through block_table[b, :]):
 *
 *   z[h,t]   = softmax_scale * (q_nope[b,h] . c_t + q_rope[b,h] . r_t)
 *   out[b,h] = sum_t softmax_t(z[h,.]) * c_t           (bf16, 512 values)
 *   lse[b,h] = log sum_t exp(z[h,t])                   (natural log, float)
 *
 * An empty V_b gives out = 0 and lse = -inf.  Arithmetic: FP16 tensor-core
 * operands (the dequantized values are exact in FP16; each head's q is
 * scaled by a power of two into [2^14, 2^15) before its bf16 -> FP16
 * conversion, the inverse folded into that head's softmax scale, so any
 * finite bf16 query is accepted) and FP32 accumulation and softmax; when
 * the list is split over several CTAs (mla_sparse_decode_plan), each split's
 * normalised partial output is rounded to FP16 in the workspace before the
 * FP32 LSE-weighted merge.
 *
 *   q_nope        device bf16 [batch, num_heads, 512] (W_UK already absorbed)
 *   q_rope        device bf16 [batch, num_heads, 64]
 *   kv_pool, kv_block_stride, num_blocks   as for mla_kv_quantize_append
 *   block_table   device int32 [batch, max_blocks_per_req]
 *   context_lens  device int32 [batch]
 *   topk_idx      device int32 [batch, topk], logical positions; any order
 *   num_heads     16, 32, 48, ..., 128
 *   topk          1..2048
 *   out           device bf16 [batch, num_heads, 512]
 *   lse           device float [batch, num_heads], or NULL
 *   workspace     device, 256-byte aligned, at least
 *                 mla_sparse_decode_workspace_size(batch, num_heads, topk)
 *                 bytes (that size depends on the current device and may be
 *                 0); contents on entry do not matter
 * batch == 0 is a no-op.
 */
size_t mla_sparse_decode_workspace_size(int batch, int num_heads, int topk);

/*
 * How mla_sparse_decode (and the FP8, no-alloc and draft-token variants, the
 * latter with batch = requests x query tokens) divides one call's work on the
 * current device.  Each (request, 16-head group) is split along its top-k
 * list into *splits CTAs of *rows_per_split entries (a multiple of 16); the
 * splits' partial outputs are combined by their LSEs.  *kernels is the number
 * of kernels the call launches: 1 for one split, or for 2..8 splits, which
 * form a thread-block cluster and merge inside the decode kernel; 2 for more
 * splits, merged by a second kernel.  Output pointers may be NULL.
 * MLA_ERR_INVALID_ARG for batch < 1, num_heads not a positive multiple of
 * 16, or topk < 1.
 *
 * The plan describes the 16-head kernel.  An NVFP4 call whose num_heads is a
 * multiple of 64 and whose pool stride is a whole number of 352-byte rows
 * runs the tensor-memory kernel instead: one CTA per (request, 64-head
 * block) and split, min(SMs / blocks, ceil(topk / 128), *splits) splits of
 * equal length (at least 1), merged by a second kernel when there are
 * several.  The workspace size covers both.
 */
mla_status_t mla_sparse_decode_plan(int batch, int num_heads, int topk, int* splits, int* rows_per_split,
                                    int* kernels);

/*
 * The division a call with this cache format and pool geometry actually
 * uses: as mla_sparse_decode_plan, and *tensor_memory = 1 when the call runs
 * the tensor-memory kernel (fmt MLA_KV_NVFP4, num_heads a multiple of 64,
 * kv_block_stride a whole number of 352-byte rows, num_blocks > 0 and fewer
 * than 2^31 pool rows; the pool base 16-byte aligned, as every call
 * requires).  Its splits are then per (request, 64-head block) with
 * ceil(topk / splits) rows each, and *kernels is 2 when a merge follows.
 * Output pointers may be NULL.  MLA_ERR_INVALID_ARG for an unknown fmt or
 * the arguments mla_sparse_decode_plan rejects.
 */
mla_status_t mla_sparse_decode_plan_fmt(int fmt, int batch, int num_heads, int topk, int64_t kv_block_stride,
                                        int64_t num_blocks, int* splits, int* rows_per_split, int* kernels,
                                        int* tensor_memory);
mla_status_t mla_sparse_decode(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                               int64_t kv_block_stride, int64_t num_blocks, const int32_t* block_table,
                               int max_blocks_per_req, const int32_t* context_lens, const int32_t* topk_idx,
                               int batch, int num_heads, int block_size, int topk, float softmax_scale,
                               uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                               mla_stream_t stream);

/*
 * Allocation-free variant of mla_sparse_decode (NVFP4 cache).  The pages
 * describe no such entry point; it exists for callers that cannot allocate
 * device memory when they call the decode: a serving process that reserves
 * its whole device-memory budget at start-up and may not grow it afterwards,
 * or a plain C host that embeds this library without a device allocator of
 * its own.  Those callers still own and pass every input and output buffer;
 * only the split-K scratch moves into the library.
 *
 *  - Arguments, results and errors are those of mla_sparse_decode, without
 *    the workspace pair.
 *  - The scratch is one file-scope device array of
 *    MLA_SPARSE_DECODE_NOALLOC_SCRATCH_BYTES (16 MiB) that every GPU which
 *    loads the library holds until the process exits.  A call whose
 *    mla_sparse_decode_workspace_size(batch, num_heads, topk) exceeds it
 *    returns MLA_ERR_WORKSPACE_TOO_SMALL and launches nothing.
 *  - The first call on a device looks up that device's address of the array
 *    (with the device current) and caches it; make that first call before any
 *    stream capture.  The call itself never calls cudaMalloc or cudaFree.
 *    The cached address does not survive cudaDeviceReset (the array may be
 *    placed elsewhere when the library's module is loaded again): a process
 *    that resets a device must not call this entry point on it afterwards.
 *  - Every call on a device shares the same array, which keeps whatever the
 *    last call left there (nothing in it needs to start at zero).  Calls that
 *    overlap on the GPU -- on different streams, or from different host
 *    threads -- race on it and must be serialised by the caller.
 */
#define MLA_SPARSE_DECODE_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)
mla_status_t mla_sparse_decode_noalloc(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                                       int64_t kv_block_stride, int64_t num_blocks, const int32_t* block_table,
                                       int max_blocks_per_req, const int32_t* context_lens, const int32_t* topk_idx,
                                       int batch, int num_heads, int block_size, int topk, float softmax_scale,
                                       uint16_t* out, float* lse, mla_stream_t stream);

/* The same decode over the 576-byte FP8 cache: c_t and r_t are the e4m3
 * bytes themselves.  This is the in-library comparison path ("Prime
 * Inference", figure "staged vs native decode": FP8 attention on a real FP8
 * cache).  Identical arguments and workspace size. */
mla_status_t mla_sparse_decode_fp8(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                                   int64_t kv_block_stride, int64_t num_blocks, const int32_t* block_table,
                                   int max_blocks_per_req, const int32_t* context_lens, const int32_t* topk_idx,
                                   int batch, int num_heads, int block_size, int topk, float softmax_scale,
                                   uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                                   mla_stream_t stream);

/*
 * Several query tokens per request, decoded in one launch (speculative draft
 * tokens: "Prime Inference", section "A kernel that reads four bits
 * directly" -- the native kernel handles 15 query tokens in one launch).  Each
 * query token has its own top-k list; the q_len tokens of request b are the
 * last q_len positions of its context_lens[b] tokens, so token i sees only
 * t < context_lens[b] - (q_len - 1 - i) (entries at or past that bound are
 * masked like any out-of-context entry).  Otherwise the decode of each token
 * is exactly that of mla_sparse_decode (fmt MLA_KV_NVFP4) or
 * mla_sparse_decode_fp8 (fmt MLA_KV_FP8).
 *
 *   q_nope        device bf16 [batch, q_len, num_heads, 512]
 *   q_rope        device bf16 [batch, q_len, num_heads, 64]
 *   topk_idx      device int32 [batch, q_len, topk]
 *   q_len         1..64
 *   out           device bf16 [batch, q_len, num_heads, 512]
 *   lse           device float [batch, q_len, num_heads], or NULL
 *   workspace     at least mla_sparse_decode_mtp_workspace_size(batch,
 *                 q_len, num_heads, topk) bytes, 256-byte aligned
 * All other arguments as for mla_sparse_decode.
 */
size_t mla_sparse_decode_mtp_workspace_size(int batch, int q_len, int num_heads, int topk);
mla_status_t mla_sparse_decode_mtp(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                                   int64_t kv_block_stride, int64_t num_blocks, const int32_t* block_table,
                                   int max_blocks_per_req, const int32_t* context_lens, const int32_t* topk_idx,
                                   int batch, int q_len, int num_heads, int block_size, int topk, float softmax_scale,
                                   mla_kv_format_t fmt, uint16_t* out, float* lse, void* workspace,
                                   size_t workspace_bytes, mla_stream_t stream);

/*
 * Staged path, kept as an ablation of the native decode ("Prime Inference",
 * section "A kernel that reads four bits directly", figure "staged vs native
 * decode": the first version gathered the selected NVFP4 rows, wrote an FP8
 * copy of each to GPU memory and ran the FP8 attention kernel on the copy,
 * moving 352 + 576 + 576 bytes per selected row instead of 352).
 *
 * mla_stage_rows_fp8 is the gather step.  For request b and list entry j
 * with token t = topk_idx[b, j], valid exactly when mla_sparse_decode would
 * use it, the 576-byte FP8 row holding e4m3_rn_satfinite(e2m1 x S) for each
 * latent value and the row's 64 rope bytes unchanged is written at
 *   staged_pool + (b * nblk * 64 + j) * 576,   nblk = ceil(topk / 64),
 * and staged_topk[b, j] = j; a masked entry writes staged_topk[b, j] = -1
 * and no row.  With block table [b, i] = b * nblk + i and context length
 * nblk * 64, the staged pool is an ordinary FP8 pool (block stride
 * 64 * 576) for mla_sparse_decode_fp8 with staged_topk as its list.
 *
 *   kv_pool ... topk   as for mla_sparse_decode (NVFP4 pool)
 *   staged_pool   device, 16-byte aligned, mla_staged_pool_bytes(batch, topk)
 *   staged_topk   device int32 [batch, topk]
 *
 * mla_sparse_decode_staged runs both steps (the gather, then the FP8 decode)
 * with every intermediate in `workspace`; its arguments and results are those
 * of mla_sparse_decode, and its outputs differ from the native decode's only
 * by the e4m3 rounding of the staged copy.
 */
size_t mla_staged_pool_bytes(int batch, int topk);
mla_status_t mla_stage_rows_fp8(const void* kv_pool, int64_t kv_block_stride, int64_t num_blocks,
                                const int32_t* block_table, int max_blocks_per_req, const int32_t* context_lens,
                                const int32_t* topk_idx, int batch, int block_size, int topk, void* staged_pool,
                                int32_t* staged_topk, mla_stream_t stream);
size_t mla_sparse_decode_staged_workspace_size(int batch, int num_heads, int topk);
mla_status_t mla_sparse_decode_staged(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                                      int64_t kv_block_stride, int64_t num_blocks, const int32_t* block_table,
                                      int max_blocks_per_req, const int32_t* context_lens, const int32_t* topk_idx,
                                      int batch, int num_heads, int block_size, int topk, float softmax_scale,
                                      uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                                      mla_stream_t stream);

/*
 * Exact top-k over float scores ("GLM-5.3 PCP/DCP long-context on H200",
 * section 1: attention reads only the 2,048 tokens the indexer rates best).
 * For request b the candidates are t in [0, min(context_lens[b],
 * max_context_len)), ordered by (score descending, t ascending), with -0.0
 * equal to +0.0; the first min(k, n) are written to topk_out[b, :] in
 * ascending t, and the rest of the row is -1.  NaN scores are not supported.
 *
 *   scores        device float, request b at scores + b * score_row_stride
 *   topk_out      device int32 [batch, topk]
 *   topk          1..2048
 *   workspace     device, 256-byte aligned, at least
 *                 mla_topk_workspace_size(...) bytes (candidate lists of
 *                 the parallel collection pass); contents on entry do not
 *                 matter
 */
size_t mla_topk_workspace_size(int batch, int max_context_len, int topk);
mla_status_t mla_topk(const float* scores, int64_t score_row_stride, const int32_t* context_lens, int batch,
                      int topk, int max_context_len, int32_t* topk_out, void* workspace, size_t workspace_bytes,
                      mla_stream_t stream);

/*
 * Indexer score plus exact top-k.  For request b and t < context_lens[b]:
 *
 *   score[b,t] = sum_h head_w[b,h] * max(0, s_t * (q_idx[b,h] . k_t))
 *
 * where k_t is the token's 128 e4m3 key values and s_t its float scale
 * ("GLM-5.3 PCP/DCP long-context on H200", section 3: a key is 128 e4m3
 * bytes and a float scale); then topk_out = mla_topk(score).  The products
 * run on the tensor cores with FP32 accumulation.  Each head's query is
 * first scaled by a power of two 2^k_h and its weight by 2^-k_h (exact:
 * relu is positively homogeneous), so any finite bf16 query is accepted.
 * With 32 or 64 index heads and a block stride that is a multiple of 128
 * bytes the operands are e4m3: the keys as stored, the query scaled into
 * [128, 256) and split into two e4m3 parts (an element is represented to
 * within max|q_h| 2^-17).  Otherwise they are FP16: the keys exact, the
 * query scaled into [2^14, 2^15) (exact for elements above 2^-10 of the
 * head's largest, FP16 subnormals below that).
 *
 *   q_idx         device bf16 [batch, n_idx_heads, 128]
 *   head_w        device float [batch, n_idx_heads]
 *   idx_key_pool  device, 16-byte aligned; block b at idx_key_pool +
 *                 b * idx_block_stride holds block_size x 128 key bytes
 *                 followed by block_size float scales
 *   idx_block_stride  bytes, a multiple of 16, >= block_size * 132
 *   n_idx_heads   8, 16, 32 or 64 (other multiples of 8 up to 64 return
 *                 MLA_ERR_UNSUPPORTED, anything else MLA_ERR_INVALID_ARG)
 *   topk_out      device int32 [batch, topk]
 *   scores_out    device float [batch, max_context_len] (entries past a
 *                 request's context are left untouched), or NULL to keep
 *                 the scores in the workspace only
 *   max_context_len  >= every context_lens[b] that should be fully scored;
 *                 longer contexts are cut to it
 */
size_t mla_indexer_topk_workspace_size(int batch, int max_context_len, int topk);
mla_status_t mla_indexer_topk(const uint16_t* q_idx, const float* head_w, const void* idx_key_pool,
                              int64_t idx_block_stride, int64_t num_blocks, const int32_t* block_table,
                              int max_blocks_per_req, const int32_t* context_lens, int batch, int n_idx_heads,
                              int block_size, int topk, int32_t* topk_out, float* scores_out, int max_context_len,
                              void* workspace, size_t workspace_bytes, mla_stream_t stream);

/*
 * Block tables and slot maps from request lengths, built on the device.
 * Request b holds context_lens[b] tokens in its first ceil(context_lens[b] /
 * block_size) blocks and gets new_lens[b] more (0 for one that waits; a
 * negative length counts as 0).  The blocks that it then lacks are taken from
 * a ring of free block ids, request by request and in order, and written
 * behind its last one in its row of the block table; every new token's
 * position and slot follow:
 *
 *   query_start[b] = sum of new_lens before b, query_start[batch] = their sum
 *   positions[query_start[b] + j]    = context_lens[b] + j
 *   slot_mapping[query_start[b] + j] = block * block_size + position % block_size
 *
 * as the quantize-on-write entry points read them.  Entries behind the last
 * token are -1 in both, so a call captured at a fixed num_slots serves any
 * smaller number of tokens.  Tokens past num_slots are left out: they count
 * in no output.
 *
 * The ring's entries free_state[0] (head) to free_state[1] (tail) - 1, each
 * taken modulo free_capacity, are the free blocks; a call takes from the head
 * and the caller returns blocks at the tail.  When it runs short, what is
 * left goes to the first requests: a block that could not be had is -1 in
 * the table, its tokens' slots are -1, and context_lens_out counts a
 * request's tokens up to the first such block only.  The same holds for
 * tokens past max_blocks_per_req blocks.  An entry of the table or the ring
 * outside [0, num_blocks) gives its tokens slot -1.
 *
 *   context_lens      device int32 [batch], new_lens device int32 [batch]
 *   block_table       device int32 [batch, max_blocks_per_req], in and out:
 *                     only entries of new blocks are written
 *   free_blocks       device int32 [free_capacity]
 *   free_state        device int64 [3]: head, tail (the third is not read)
 *   slot_mapping      device int64 [num_slots], positions int32 [num_slots]
 *   query_start       device int32 [batch + 1]
 *   context_lens_out  device int32 [batch]; may be context_lens
 *   free_state_out    device int64 [3]: head past the blocks taken, tail,
 *                     blocks that could not be had; may be free_state
 * No other two arguments may overlap.
 */
mla_status_t mla_block_table_extend(const int32_t* context_lens, const int32_t* new_lens, int batch,
                                    int32_t* block_table, int max_blocks_per_req, const int32_t* free_blocks,
                                    int64_t free_capacity, const int64_t* free_state, int64_t num_blocks,
                                    int block_size, int64_t* slot_mapping, int32_t* positions, int64_t num_slots,
                                    int32_t* query_start, int32_t* context_lens_out, int64_t* free_state_out,
                                    mla_stream_t stream);

/*
 * Norms of queries and keys for each head, with the position rotation in the
 * same pass.  For every token and head, x its head_dim values:
 *
 *   y = x / sqrt(mean(x^2) + eps) * weight      (y = x without a weight)
 *   the 64 values of y from rope_offset on are rotated in pairs by the angle
 *   positions[token] * inv_freq[i], i = 0..31:
 *   (y0, y1) -> (y0 cos - y1 sin, y1 cos + y0 sin)
 *
 * where pair i is values 2i and 2i + 1 (interleaved nonzero) or i and i + 32.
 * Float32 arithmetic, one rounding to bf16 at the end.  The angle is kept as a
 * 64-bit fraction of a turn: for inv_freq up to 1 it is within 2^-31 +
 * |position| x 2^-55 of a turn.
 *
 *   q, k          head sets on the host, either may be NULL (or have 0 heads)
 *     in, out     device bf16, 16-byte aligned; head h of token t starts at
 *                 t * token stride + h * head stride (elements, multiples of
 *                 8; that of an axis with one entry is not used); out may
 *                 be in with the same strides, else no element of one may be
 *                 in the other; no two heads of out may share an element
 *                 (checked), nor the outputs of q and k
 *     weight      device bf16 [head_dim], 16-byte aligned, or NULL: no norm
 *   head_dim      64..256, a multiple of 8 (wider: MLA_ERR_UNSUPPORTED)
 *   rope_offset   0..head_dim - 64, a multiple of 8
 *   eps           > 0
 *   positions     device int32 [n_tokens]
 *   inv_freq      device double [32], radians per position
 * n_tokens == 0 is a no-op.
 */
typedef struct {
  const uint16_t* in;
  uint16_t* out;
  int heads;
  int64_t in_token_stride, in_head_stride, out_token_stride, out_head_stride;
  const uint16_t* weight;
} mla_heads_t;
mla_status_t mla_qk_norm_rope(const mla_heads_t* q, const mla_heads_t* k, int64_t n_tokens, int head_dim,
                              int rope_offset, int interleaved, float eps, const int32_t* positions,
                              const double* inv_freq, mla_stream_t stream);

/*
 * The same pass for a step of the cache: each token's latent is normed, its
 * 64 key values are rotated, and the row is quantised into the paged cache,
 * without a bf16 copy of it in memory; the queries' norms and rotation (q, as
 * above, or NULL) run in the same launch.  The normed latent and the rotated
 * key are rounded to bf16 before they are quantised, so the cache holds the
 * bytes that mla_kv_quantize_append writes for those bf16 rows.
 *
 *   kv            device bf16 [n_tokens, 512 latent + 64 key], 16-byte
 *                 aligned, rows kv_token_stride elements apart (a multiple
 *                 of 8; not used with one token)
 *   latent_weight device bf16 [512], 16-byte aligned
 *   slot_mapping, kv_pool, num_blocks, block_size, kv_block_stride, fmt
 *                 as for mla_kv_quantize_append
 *   head_dim, rope_offset   of q (ignored without q)
 * n_tokens == 0 is a no-op.  Two tokens with the same slot race.
 */
mla_status_t mla_kv_norm_rope_append(const uint16_t* kv, int64_t kv_token_stride, const uint16_t* latent_weight,
                                     const mla_heads_t* q, int head_dim, int rope_offset, int interleaved, float eps,
                                     const int32_t* positions, const double* inv_freq, const int64_t* slot_mapping,
                                     int64_t n_tokens, void* kv_pool, int64_t num_blocks, int block_size,
                                     int64_t kv_block_stride, mla_kv_format_t fmt, mla_stream_t stream);

/*
 * Dense decode over a sliding window and the first tokens.  The q_len query
 * tokens of request b are the last q_len positions of its context_lens[b]
 * tokens: token i stands at p = context_lens[b] - q_len + i and sees
 *
 *   { t : 0 <= t <= p  and  (t < sinks  or  t > p - window) }
 *
 * and out, lse are those of mla_sparse_decode over that set (the same
 * arithmetic; rows whose logical block is past the table or whose physical
 * block is outside the pool are not seen; a token that sees nothing gives 0
 * and -inf).  A window of at least the context is a decode over all of it.
 * Every row that a token of the call sees is read once per 64 (query token,
 * head) pairs of its request.  The weights of the rows in out are FP16 operands:
 * each is off by at most 2^-11 of itself, or by 2^-34 of the query's largest
 * weight in the same slice where that is more (rows 2^23 below it and further);
 * the slices' partial outputs are float.
 *
 *   q_nope        device bf16 [batch, q_len, num_heads, 512]
 *   q_rope        device bf16 [batch, q_len, num_heads, 64], 16-byte aligned
 *   q_len         1..64
 *   sinks >= 0, window >= 1
 *   out           device bf16 [batch, q_len, num_heads, 512]
 *   lse           device float [batch, q_len, num_heads], or NULL
 *   workspace     at least mla_window_decode_workspace_size(...) bytes,
 *                 256-byte aligned (that size depends on the current device
 *                 and may be 0); contents on entry do not matter; calls that
 *                 may run at the same time need one each
 * All other arguments as for mla_sparse_decode.  batch == 0 is a no-op.
 */
size_t mla_window_decode_workspace_size(int batch, int q_len, int num_heads, int max_blocks_per_req, int sinks,
                                        int window);
mla_status_t mla_window_decode(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                               int64_t kv_block_stride, int64_t num_blocks, const int32_t* block_table,
                               int max_blocks_per_req, const int32_t* context_lens, int batch, int q_len,
                               int num_heads, int block_size, int sinks, int window, float softmax_scale,
                               mla_kv_format_t fmt, uint16_t* out, float* lse, void* workspace,
                               size_t workspace_bytes, mla_stream_t stream);

/*
 * Dense decode of requests that share a prefix.  Every query token of the
 * batch sees the prefix_len rows of prefix_table and, behind them, its own
 * request's rows: token i of request b sees own rows t < context_lens[b] -
 * (q_len - 1 - i), where context_lens[b] counts the tokens after the prefix
 * (0: the prefix alone).  The prefix is walked once per 64 (request, query
 * token, head) triples of the whole batch, not once per request, and the two
 * parts are joined by their LSEs.
 *
 *   prefix_table  device int32 [ceil(prefix_len / block_size)] (not read when
 *                 prefix_len is 0)
 *   block_table   device int32 [batch, max_blocks_per_req], own blocks
 *   max_context_len  >= every context_lens[b]; longer ones are cut to it
 *   workspace     at least mla_prefix_decode_workspace_size(...) bytes,
 *                 256-byte aligned
 * All other arguments as for mla_window_decode.
 */
size_t mla_prefix_decode_workspace_size(int batch, int q_len, int num_heads, int prefix_len, int max_blocks_per_req,
                                        int max_context_len);
mla_status_t mla_prefix_decode(const uint16_t* q_nope, const uint16_t* q_rope, const void* kv_pool,
                               int64_t kv_block_stride, int64_t num_blocks, const int32_t* prefix_table,
                               int prefix_len, const int32_t* block_table, int max_blocks_per_req,
                               const int32_t* context_lens, int batch, int q_len, int num_heads, int block_size,
                               int max_context_len, float softmax_scale, mla_kv_format_t fmt, uint16_t* out,
                               float* lse, void* workspace, size_t workspace_bytes, mla_stream_t stream);

/*
 * Attention over whole prompts, packed one behind another.  Sequence b has the
 * query tokens query_start[b] .. query_start[b + 1] - 1 and the keys and values
 * kv_start[b] .. kv_start[b + 1] - 1 (nq and nk of them); its queries are the
 * last nq of its nk positions: query token i sees
 *
 *   causal      t < nk - nq + i + 1      (nothing where that is not positive)
 *   otherwise   every t < nk
 *
 *   out = sum_t softmax_t(softmax_scale * q . k_t) v_t,   lse = the natural
 *   logarithm of the softmax's denominator
 *
 * with query head h using key head h / (num_heads / num_kv_heads).  A token that
 * sees nothing gives 0 and -inf.  Prompts, their later chunks behind earlier
 * keys, drafts and single tokens are the same call.  Scores, softmax statistics
 * and sums are float32; a weight enters the product as bf16 (off by at most
 * 2^-8 of itself).  The largest score that a token sees, times softmax_scale and
 * log2 e, must be less than 2^30 in magnitude: from there on, -infinity
 * included, the token's out and lse are NaN.  What a token does not see never
 * reaches its output, be it infinite or NaN.
 *
 *   q             device bf16 [q_tokens, num_heads, qk_dim]
 *   k, v          device bf16 [kv_tokens, num_kv_heads, qk_dim / v_dim]; not
 *                 read if kv_tokens is 0
 *   out           device bf16 [q_tokens, num_heads, v_dim]; tokens before the
 *                 first sequence and behind the last are not written
 *   strides       elements, multiples of 8, less than 2^39; that of an axis with
 *                 one entry is not used; those of q, k and v at least qk_dim or
 *                 v_dim (less, also the 0 of a repeated axis:
 *                 MLA_ERR_UNSUPPORTED); no two rows of out may share an element
 *                 (checked), out may not overlap an input.  All four tensors
 *                 16-byte aligned
 *   query_start, kv_start   device int32 [batch + 1], not decreasing; values
 *                 outside [0, q_tokens] or [0, kv_tokens] are cut to it
 *   qk_dim        a multiple of 8, 8..192; v_dim 8..128 (more:
 *                 MLA_ERR_UNSUPPORTED)
 *   num_heads     a multiple of num_kv_heads, at most 128 of them for each
 *                 (more: MLA_ERR_UNSUPPORTED)
 *   softmax_scale finite, of either sign
 *   lse           device float [q_tokens, num_heads], or NULL
 *   workspace     at least mla_prompt_attention_workspace_size(...) bytes,
 *                 256-byte aligned (that size depends on the current device
 *                 and may be 0); contents on entry do not matter; calls that
 *                 may run at the same time need one each
 * batch == 0 or q_tokens == 0 is a no-op.  At most 2^31 - 256 tokens and
 * sequences, and q_tokens x num_heads and batch x num_kv_heads < 2^31 (more:
 * MLA_ERR_UNSUPPORTED).
 */
size_t mla_prompt_attention_workspace_size(int64_t q_tokens, int64_t kv_tokens, int batch, int num_heads,
                                           int num_kv_heads, int v_dim);

/*
 * How a call of these sizes is divided on the current device.  A unit is
 * *row_tiles (1 or 2) times 128 rows of one sequence and key head, with all of
 * its keys or one of *slices parts of them (several are joined by a second
 * kernel); *units is the number of CTAs in the grid: as many as the device has
 * SMs run, and take over the others' units (some of which may be empty, as
 * lengths are known on the device only).  *variant: 0 plain, 1 the
 * exponentials of a unit's two tiles take turns, 2 a unit of one filled tile has its
 * keys shared by two halves.  Output pointers may be NULL.
 */
mla_status_t mla_prompt_attention_plan(int64_t q_tokens, int64_t kv_tokens, int batch, int num_heads, int num_kv_heads,
                                       int v_dim, int* row_tiles, int* slices, int64_t* units, int* variant);
mla_status_t mla_prompt_attention(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, const uint16_t* k,
                                  int64_t k_token_stride, int64_t k_head_stride, const uint16_t* v,
                                  int64_t v_token_stride, int64_t v_head_stride, const int32_t* query_start,
                                  const int32_t* kv_start, int batch, int64_t q_tokens, int64_t kv_tokens,
                                  int num_heads, int num_kv_heads, int qk_dim, int v_dim, int causal,
                                  float softmax_scale, uint16_t* out, int64_t out_token_stride,
                                  int64_t out_head_stride, float* lse, void* workspace, size_t workspace_bytes,
                                  mla_stream_t stream);

/*
 * The residual's addition, the norm behind it, and its output in 8 bits.  For
 * every row of dim values:
 *
 *   h = x + residual                    (h = x without one)
 *   y = h / sqrt(mean(h^2) + eps) * weight
 *   scales[g] = max |y_i| / 448  over group g,   codes[i] = e4m3(y_i / scales[g])
 *
 * in float32, e4m3 rounded to nearest even.  h is rounded only where it is
 * stored, in the residual's type: the norm is that of the sum before.  Groups
 * are 128 values (the last one what is left) or the row.  A group of zeros has
 * scale 0 and codes 0; one that holds a NaN or whose y does has scale NaN.
 * Squares past float32's range do not matter; sums h past it are infinite.
 *
 *   x               device bf16, 16-byte aligned, rows x_stride elements
 *                   apart (a multiple of 8; strides are not used with one row)
 *   residual_type   MLA_RESIDUAL_NONE (residual and residual_out are not
 *                   used), _BF16 or _F32
 *   residual        device, 16-byte aligned, rows residual_stride elements
 *                   apart (16 bytes' multiple)
 *   residual_out    likewise; may be residual with the same stride, else
 *                   no element of it may be in another argument
 *   weight          device bf16 [dim], 16-byte aligned
 *   dim             a multiple of 8, 8..16384 (more: MLA_ERR_UNSUPPORTED)
 *   group           128, or 0: the row (others: MLA_ERR_UNSUPPORTED)
 *   eps             > 0
 *   codes           device e4m3 [n_tokens, dim], 8-byte aligned
 *   scales          device float [n_tokens, ceil(dim / group) or 1]
 * n_tokens == 0 is a no-op.
 */
typedef enum { MLA_RESIDUAL_NONE = 0, MLA_RESIDUAL_BF16 = 1, MLA_RESIDUAL_F32 = 2 } mla_residual_t;
mla_status_t mla_add_norm_quant(const uint16_t* x, int64_t x_stride, mla_residual_t residual_type,
                                const void* residual, int64_t residual_stride, void* residual_out,
                                int64_t residual_out_stride, const uint16_t* weight, int64_t n_tokens, int dim,
                                int group, float eps, uint8_t* codes, float* scales, mla_stream_t stream);

/*
 * Products of a few tokens with matrices of 4-bit weights, one for each of
 * `groups` (1: a projection of the token; the heads: each head's own):
 *
 *   out[t,g,n] = weight_scale[g] * sum_k x[t,g,k] * code[g,n,k] * scale[g,n,k/16]
 *
 * with the format of the cached latents: e2m1 codes, element 2i in the low
 * nibble of byte i, and one e4m3 scale per 16.  x is bf16, or e4m3 codes with
 * float scales as mla_add_norm_quant writes them.  Products are exact f16
 * operands added up in float32 (a bf16 x loses what lies 2^-39 below the largest of
 * its 128); the same call gives the same bits.  The weights are read once for
 * up to 32 tokens (more tokens: once per 32).
 *
 *   x               device bf16 or e4m3, 16-byte aligned; group g of token t
 *                   starts at t * token stride + g * group stride (elements,
 *                   16 bytes' multiples; that of an axis with one entry is
 *                   not used)
 *   x_scales        device float [n_tokens, groups, x_scale_groups] (e4m3 only)
 *   x_scale_groups  ceil(k / 128): one per 128 values; or 1: one per row
 *   codes           device [groups, n, k / 2] bytes, 16-byte aligned
 *   scales          device e4m3 [groups, n, k / 16], 2-byte aligned
 *   weight_scale    device float [groups], or NULL: 1
 *   k               a multiple of 32 (odd multiples of 16: MLA_ERR_UNSUPPORTED)
 *   out             device bf16 or float, strides as x's, in elements (any);
 *                   no two rows may share an element (checked), nor may
 *                   they overlap another argument
 *   groups          at most 65,535; n_tokens at most 2,097,120 (more:
 *                   MLA_ERR_UNSUPPORTED)
 * n_tokens, groups or n == 0 is a no-op.
 */
typedef enum { MLA_X_BF16 = 0, MLA_X_E4M3 = 1 } mla_x_type_t;
typedef enum { MLA_OUT_BF16 = 0, MLA_OUT_F32 = 1 } mla_out_type_t;
mla_status_t mla_fp4_matvec(const void* x, mla_x_type_t x_type, int64_t x_token_stride, int64_t x_group_stride,
                            const float* x_scales, int x_scale_groups, const uint8_t* codes, const uint8_t* scales,
                            const float* weight_scale, int64_t n_tokens, int groups, int n, int k, void* out,
                            mla_out_type_t out_type, int64_t out_token_stride, int64_t out_group_stride,
                            mla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_NVFP4_H */
