// Dense MLA decode over the paged cache on the fifth-generation tensor cores:
// a sliding window with first tokens that stay visible, and a batch whose
// requests share a prefix.  NVFP4 or FP8 rows, f16 operands, f32 accumulation.
//
// Mathematics.  64 "columns" -- (query token, head) pairs that look at the
// same cached rows -- share one walk over those rows in tiles of 128:
//   S[128 rows x 64 columns] = K[128 x 576] . Q^T
//   P = 2^(S scale - m), m the column's running maximum (raised lazily)
//   O^T[512 x 64] = O^T + V^T[512 x 128] . P,   V = the first 512 of K
// and each column's denominator is summed in float beside it, so the rows are
// read and unpacked once for all 64 columns.  A request's query tokens and
// heads fill columns; where the rows are a shared prefix, so do the requests.
//
// Work split.  One CTA = 64 columns x a slice of their rows; slices' partial
// outputs (normalised, f16) and base-2 LSEs are joined by dense_merge_kernel.
// 16 warps unpack (a row's 16-byte pieces straight from global memory into
// registers, one tile ahead), run the softmax and write the output; the
// 17th issues every tcgen05.mma.  The unpacked tile is stored once, as 8 x 8
// core matrices, dim group major, which is at the same time the K-major A
// operand of S (M = 128 rows) and the MN-major A operand of O^T (M = 128
// dims).  There is room for one tile (144 KB) beside the query (72 KB), so it
// is handed over in five regions (4 x 128 latent dims, rope): a region is
// refilled with the next tile as soon as the O^T product has left it, while
// that product works on the regions after it, and S of the next tile starts
// on the regions already filled.  P lies in the rope region, which only S
// reads.
//
// Every wait is bounded; one that runs out sets the library's fault bit and
// the CTA leaves after its MMAs in flight have drained.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kRows = 128;  // rows per tile
constexpr int kCols = 64;   // columns per CTA
constexpr int kWarps = 16;  // unpack / softmax warps
constexpr int kComputeThreads = kWarps * 32;
constexpr int kThreads = kComputeThreads + 32;     // + the MMA warp
constexpr int kDimGroups = (kLatent + kRope) / 8;  // 72
constexpr int kDgBytes = kRows * 16;               // one 8-dim group of a tile: 2,048
constexpr int kTileBytes = kDimGroups * kDgBytes;  // 147,456
constexpr int kPOff = kLatent / 8 * kDgBytes;      // P overlays the rope region
constexpr int kQGroupBytes = kDimGroups * 128;     // 8 columns x 576 dims: 9,216
constexpr int kQBytes = kCols / 8 * kQGroupBytes;  // 73,728
constexpr int kRegions = 5;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 64;  // S: columns 0-63, O^T: 64-319
// The maximum of a column is raised only when a score exceeds it by 2^8: P
// stays within 2^8 in f16 and O^T is rarely rescaled.
constexpr float kLazyRaise = 8.f;
constexpr float kLn2f = 0.6931471805599453f;

struct alignas(1024) Smem {
  uint8_t tile[kTileBytes];  // (dim / 8) * 2048 + row * 16 + (dim % 8) * 2
  uint8_t q[kQBytes];        // (col / 8) * 9216 + (dim / 8) * 128 + (col % 8) * 16
  float red[kWarps][16];     // per warp, per column reduction scratch
  float m_ref[kCols];        // running (lazy) maximum, base 2
  float alpha[kCols];        // factor of the last raise; at the end 1 / denominator
  float qscale[kCols];       // softmax scale (base 2) x 2^-shift of the column's query
  uint32_t qmax[kCols];      // largest |q| of the column (bf16 magnitude bits)
  uint64_t full[kRegions], free_[kRegions], s_full, p_full, done;
  uint32_t tmem_base;
  int abort_flag;  // set by whoever ran out of polls; ends the others' waits
  int abort_tile;  // first tile whose barrier an unpack warp reached with a failed wait
};
static_assert(sizeof(Smem) <= 227 * 1024, "one CTA per SM must fit");

// ---- tcgen05 operands ---------------------------------------------------------
// No-swizzle shared-memory descriptor: start, byte offset between core
// matrices along K, and along M / N (all >> 4), descriptor version 1.
__device__ __forceinline__ uint64_t op_desc(uint32_t saddr, uint32_t k_stride, uint32_t mn_stride) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(k_stride >> 4) << 16) |
         (static_cast<uint64_t>(mn_stride >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}
// kind::f16, f16 operands, f32 accumulator, M = 128; majorness 1 = MN-major.
__device__ __forceinline__ uint32_t f16_idesc(int n, uint32_t a_mn, uint32_t b_mn) {
  return (1u << 4) | (a_mn << 15) | (b_mn << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void umma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// OR of `pred` over the unpack warps (named barrier 2).
__device__ __forceinline__ bool compute_any(bool pred) {
  uint32_t out;
  asm volatile(
      "{ .reg .pred pi, po; setp.ne.u32 pi, %1, 0; barrier.cta.red.or.pred po, 2, %2, pi; selp.u32 %0, 1, 0, po; }"
      : "=r"(out)
      : "r"(static_cast<uint32_t>(pred)), "r"(kComputeThreads)
      : "memory");
  return out != 0;
}
__device__ __forceinline__ bool wait_bar(Smem& sm, uint64_t* bar, uint32_t parity, unsigned int* fw) {
  if (mbar_try_wait(bar, parity)) return true;
  if (mbar_wait_or_abort(bar, parity, &sm.abort_flag, fw, kFaultDecodeWait)) return true;
  *reinterpret_cast<volatile int*>(&sm.abort_flag) = 1;
  return false;
}
// The same for a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool wait_bar_warp(Smem& sm, uint64_t* bar, uint32_t parity, unsigned int* fw) {
  return __all_sync(0xFFFFFFFFu, wait_bar(sm, bar, parity, fw));
}
// One arrival per warp after all its lanes' shared-memory writes: each lane
// publishes its own writes to the tensor core's proxy first.
__device__ __forceinline__ void warp_publish(uint64_t* bar, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Reduction over the 32 lanes of 16 per-lane values (one per column): lane l
// ends with column l / 2 (both lanes of a pair hold it).  Halving exchange: 16
// shuffles instead of 80.
template <typename Op>
__device__ __forceinline__ float reduce_cols(float (&v)[16], int lane, Op op) {
#pragma unroll
  for (int n = 8, off = 16; n >= 1; n >>= 1, off >>= 1) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n];
      const float keep = up ? v[i + n] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, give, off));
    }
  }
  return op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 1));
}

// This thread's pieces of one row: 32 dims of each 128-dim region and 16 rope
// dims, as stored.
template <int FMT>
struct RawRow;
template <>
struct RawRow<0> {
  static constexpr int kRowBytes = kRowNvfp4;
  uint4 code[4];
  uint32_t scale[4];  // two e4m3 scales each
  uint4 rope;
  __device__ __forceinline__ void load_region(const uint8_t* row, int m, int quarter) {
    if (row != nullptr) {
      code[m] = __ldg(reinterpret_cast<const uint4*>(row + 64 * m + 16 * quarter));
      scale[m] = __ldg(reinterpret_cast<const unsigned short*>(row + kScaleOff + 8 * m + 2 * quarter));
    } else {
      code[m] = make_uint4(0, 0, 0, 0);
      scale[m] = 0;
    }
  }
  __device__ __forceinline__ void load_rope(const uint8_t* row, int quarter) {
    rope = row != nullptr ? __ldg(reinterpret_cast<const uint4*>(row + kRopeOffNvfp4 + 16 * quarter))
                          : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void unpack_region(int m, uint32_t (&h)[4][4]) const {
    const uint32_t w[4] = {code[m].x, code[m].y, code[m].z, code[m].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t s2 = e4m3x2_to_f16x2(((scale[m] >> (8 * (i >> 1))) & 0xFFu) * 0x0101u);
      e2m1x8_to_f16x2x4(w[i], h[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) h[i][k] = hmul2(h[i][k], s2);
    }
  }
};
template <>
struct RawRow<1> {
  static constexpr int kRowBytes = kRowFp8;
  uint4 code[4][2];
  uint4 rope;
  __device__ __forceinline__ void load_region(const uint8_t* row, int m, int quarter) {
    if (row != nullptr) {
      const uint4* p = reinterpret_cast<const uint4*>(row + 128 * m + 32 * quarter);
      code[m][0] = __ldg(p);
      code[m][1] = __ldg(p + 1);
    } else {
      code[m][0] = code[m][1] = make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void load_rope(const uint8_t* row, int quarter) {
    rope = row != nullptr ? __ldg(reinterpret_cast<const uint4*>(row + kRopeOffFp8 + 16 * quarter))
                          : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void unpack_region(int m, uint32_t (&h)[4][4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = code[m][i >> 1];
      uint32_t lo[2], hi[2];
      e4m3x4_to_f16x2x2((i & 1) ? v.z : v.x, lo);
      e4m3x4_to_f16x2x2((i & 1) ? v.w : v.y, hi);
      h[i][0] = lo[0];
      h[i][1] = lo[1];
      h[i][2] = hi[0];
      h[i][3] = hi[1];
    }
  }
};
__device__ __forceinline__ void unpack_rope(const uint4 v, uint32_t (&h)[2][4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo[2], hi[2];
    e4m3x4_to_f16x2x2(w[2 * i], lo);
    e4m3x4_to_f16x2x2(w[2 * i + 1], hi);
    h[i][0] = lo[0];
    h[i][1] = lo[1];
    h[i][2] = hi[0];
    h[i][3] = hi[1];
  }
}

// One CTA's work: columns [col0, col0 + ncols) over rows [begin, end) of a row
// list.  List entry j is position j for j < n_sink, else w0 + j - n_sink.
struct Unit {
  int64_t col0;
  int ncols;
  int part;  // slot of its partial among a column's
  const int32_t* table;
  int table_len;
  int n_sink, w0, begin, end;
  int tok_col0;  // col0 within its request (own rows)
  int me0;       // position of query token 0 (own rows)
  bool masked;   // own rows: visibility depends on the query token
};

__device__ __forceinline__ Unit find_unit(const DenseArgs& a) {
  Unit u;
  const int id = blockIdx.x;
  const int n_prefix = a.prefix_groups * a.prefix_splits;
  int n_rows, sp, splits;
  u.tok_col0 = u.me0 = 0;
  if (id < n_prefix) {
    sp = id % a.prefix_splits;
    splits = a.prefix_splits;
    u.col0 = static_cast<int64_t>(id / a.prefix_splits) * kCols;
    u.ncols = static_cast<int>(min(static_cast<int64_t>(kCols), a.columns - u.col0));
    u.part = sp;
    u.table = a.prefix_table;
    u.table_len = (a.prefix_len + kBlock - 1) / kBlock;
    u.n_sink = 0;
    u.w0 = 0;
    n_rows = a.prefix_len;
    u.masked = false;
  } else {
    const int v = id - n_prefix;
    sp = v % a.splits;
    splits = a.splits;
    const int g = v / a.splits;
    const int b = g / a.groups_per_req;
    u.tok_col0 = (g - b * a.groups_per_req) * kCols;
    const int req_cols = a.q_len * a.num_heads;
    u.col0 = static_cast<int64_t>(b) * req_cols + u.tok_col0;
    u.ncols = min(kCols, req_cols - u.tok_col0);
    u.part = a.prefix_splits + sp;
    u.table = a.block_table + static_cast<int64_t>(b) * a.max_blocks;
    u.table_len = a.max_blocks;
    u.masked = true;
    const int ctx = min(max(__ldg(a.ctx_lens + b), 0), a.max_context);
    u.me0 = ctx - a.q_len;
    const int me_lo = u.me0 + u.tok_col0 / a.num_heads;
    const int me_hi = u.me0 + (u.tok_col0 + u.ncols - 1) / a.num_heads;
    // positions past the table have no rows (a wrong context length must not
    // cost a walk over them)
    const int64_t held = min(static_cast<int64_t>(a.max_blocks) * kBlock, static_cast<int64_t>(0x7FFFFF00));
    const int stop = static_cast<int>(min(static_cast<int64_t>(me_hi) + 1, held));
    u.n_sink = max(0, min(a.sinks, stop));
    u.w0 = max(a.sinks, me_lo - a.window + 1);
    n_rows = u.n_sink + max(0, stop - u.w0);
  }
  // whole tiles, spread evenly over the splits
  const int tiles = (n_rows + kRows - 1) / kRows;
  const int lo = static_cast<int>(static_cast<int64_t>(tiles) * sp / splits);
  const int hi = static_cast<int>(static_cast<int64_t>(tiles) * (sp + 1) / splits);
  u.begin = lo * kRows;
  u.end = min(n_rows, hi * kRows);
  return u;
}
__device__ __forceinline__ int list_pos(const Unit& u, int j) { return j < u.n_sink ? j : u.w0 + (j - u.n_sink); }
// Physical block of list entry j, -1 if there is none (past the slice, past
// the table or outside the pool).
__device__ __forceinline__ int list_block(const DenseArgs& a, const Unit& u, int j) {
  if (j >= u.end) return -1;
  const int blk = list_pos(u, j) / kBlock;
  if (blk >= u.table_len) return -1;
  const int id = __ldg(u.table + blk);
  return id < a.num_blocks ? id : -1;
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) dense_decode_kernel(const DenseArgs args) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  unsigned int* fw = args.fault_word;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Unit u = find_unit(args);
  const int n_tiles = (u.end - u.begin + kRows - 1) / kRows;
  const bool direct = args.parts == 1;
  if (n_tiles <= 0) {  // nothing to see: an empty partial, or the whole answer
    if (direct) {
      uint4* o = reinterpret_cast<uint4*>(args.out + u.col0 * kLatent);
      for (int i = threadIdx.x; i < u.ncols * (kLatent / 8); i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
    }
    for (int c = threadIdx.x; c < u.ncols; c += kThreads) {
      if (!direct) args.part_lse[(u.col0 + c) * args.parts + u.part] = -INFINITY;
      if (direct && args.lse != nullptr) args.lse[u.col0 + c] = -INFINITY;
    }
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRegions; ++i) {
      mbar_init(&sm.full[i], kWarps);
      mbar_init(&sm.free_[i], 1);
    }
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.p_full, kWarps);
    mbar_init(&sm.done, 1);
    sm.abort_flag = 0;
    sm.abort_tile = 0x7FFFFFFF;
    fence_mbar_init();
  }
  if (threadIdx.x < kCols) {
    sm.m_ref[threadIdx.x] = -INFINITY;
    sm.qmax[threadIdx.x] = 0;
  }
  if (warp == kWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tbase = sm.tmem_base;

  if (warp == kWarps) {
    // ------------------------------------------------------------ MMA issue
    if (lane == 0) {
      const uint32_t idesc_s = f16_idesc(u.ncols, 0, 0);
      const uint32_t idesc_o = f16_idesc(u.ncols, 1, 1);
      const uint32_t tile = smem_u32(sm.tile);
      const uint32_t q = smem_u32(sm.q);
      const uint32_t p = tile + kPOff;
      bool ok = true;
      for (int n = 0; n < n_tiles && ok; ++n) {
        const uint32_t par = static_cast<uint32_t>(n) & 1u;
        // S = K . Q^T, region by region as they fill (rope last)
        for (int m = 0; m < kRegions; ++m) {
          ok = wait_bar(sm, &sm.full[m], par, fw);
          if (!ok) break;
          tcgen05_fence_after();
          const int steps = m < 4 ? 8 : 4;  // 16 dims each
#pragma unroll 4
          for (int j = 0; j < steps; ++j) {
            const int dg = 16 * m + 2 * j;
            umma_f16(tbase, op_desc(tile + dg * kDgBytes, kDgBytes, 128), op_desc(q + dg * 128, 128, kQGroupBytes),
                     idesc_s, (m | j) != 0);
          }
        }
        if (!ok) break;
        umma_commit(&sm.s_full);
        ok = wait_bar(sm, &sm.p_full, par, fw);
        if (!ok) break;
        tcgen05_fence_after();
        // O^T += V^T . P, 128 dims at a time; each leaves its region free
        for (int m = 0; m < 4; ++m) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            umma_f16(tbase + kOCol + kCols * m, op_desc(tile + 16 * m * kDgBytes + 256 * j, 128, kDgBytes),
                     op_desc(p + 256 * j, 128, kDgBytes), idesc_o, (n | j) != 0);
          umma_commit(&sm.free_[m]);
        }
        umma_commit(&sm.free_[4]);  // P (the rope region) is free when all four are done
      }
      umma_commit(&sm.done);  // arrives once every MMA issued above has completed
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ unpack, softmax, output
    const int row_u = 8 * warp + (lane & 7);  // the tile row this thread unpacks, with three others
    const int quarter = lane >> 3;            // its 32 dims of each region
    const int quad = warp & 3;                // tensor-memory lanes 32 quad .. 32 quad + 31
    const int cq = warp >> 2;                 // columns 16 cq .. 16 cq + 15
    const bool has_cols = 16 * cq < u.ncols;
    const uint32_t lane_base = static_cast<uint32_t>(32 * quad) << 16;
    RawRow<FMT> raw;
    auto row_ptr = [&](int n) -> const uint8_t* {
      const int j = u.begin + n * kRows + row_u;
      const int id = list_block(args, u, j);
      return id < 0 ? nullptr
                    : args.pool + static_cast<int64_t>(id) * args.block_stride +
                          list_pos(u, j) % kBlock * RawRow<FMT>::kRowBytes;
    };
    {
      const uint8_t* row = row_ptr(0);
#pragma unroll
      for (int m = 0; m < 4; ++m) raw.load_region(row, m, quarter);
      raw.load_rope(row, quarter);
    }
    {
      // The query, bf16 -> f16 core matrices of 8 columns x 8 dims.  A warp
      // moves 8 columns x 32 dims at a time (64-byte pieces of 8 rows in,
      // conflict-free 16-byte stores out); every load is issued before the
      // first is used.  A column whose query holds an infinity or NaN enters
      // as zeros with a NaN scale: its results are NaN, its neighbours' are not.
      constexpr int kPer = (kCols / 8) * (kDimGroups / 4) / kWarps;  // 9
      const int n_tasks = (u.ncols / 8) * (kDimGroups / 4);
      uint4 x[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int task = warp + i * kWarps;
        const int64_t col = u.col0 + task / (kDimGroups / 4) * 8 + (lane & 7);
        const int dg = task % (kDimGroups / 4) * 4 + (lane >> 3);
        x[i] = make_uint4(0, 0, 0, 0);
        if (task < n_tasks)
          x[i] = dg < kLatent / 8 ? __ldg(reinterpret_cast<const uint4*>(args.q_nope + col * kLatent) + dg)
                                  : __ldg(reinterpret_cast<const uint4*>(args.q_rope + col * kRope) + (dg - kLatent / 8));
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int task = warp + i * kWarps;
        uint32_t mx = bf16x8_absmax_bits(x[i]);
        mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
        mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
        if (task < n_tasks && lane < 8) atomicMax(&sm.qmax[task / (kDimGroups / 4) * 8 + lane], mx);
      }
      named_bar_sync(1, kComputeThreads);
      if (threadIdx.x < kCols) {
        const uint32_t mx = sm.qmax[threadIdx.x];
        sm.qscale[threadIdx.x] = mx >= 0x7F80u ? __int_as_float(0x7FFFFFFF) : args.scale_log2 * pow2f(-query_shift(mx));
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int task = warp + i * kWarps;
        if (task >= n_tasks) continue;
        const int hg = task / (kDimGroups / 4);
        const int dg = task % (kDimGroups / 4) * 4 + (lane >> 3);
        const uint32_t mx = sm.qmax[hg * 8 + (lane & 7)];
        const float mul = pow2f(query_shift(mx));
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          h[k] = mx >= 0x7F80u ? 0u
                               : f32x2_to_f16x2_sat(bf16_bits_to_f32(w[k] & 0xFFFFu) * mul,
                                                    bf16_bits_to_f32(w[k] >> 16) * mul);
        *reinterpret_cast<uint4*>(sm.q + hg * kQGroupBytes + dg * 128 + (lane & 7) * 16) =
            make_uint4(h[0], h[1], h[2], h[3]);
      }
    }
    float l_part[16];  // this row's share of each column's denominator
#pragma unroll
    for (int j = 0; j < 16; ++j) l_part[j] = 0.f;
    const int me = u.me0 + (u.tok_col0 + 16 * cq) / args.num_heads;  // 16 columns share a query token
    const float* m_ref = sm.m_ref + 16 * cq;
    const float* qscale = sm.qscale + 16 * cq;
    bool aborted = false;
    for (int n = 0; n < n_tiles; ++n) {
      const uint32_t par = static_cast<uint32_t>(n) & 1u;
      bool ok = true;
      const uint8_t* next = n + 1 < n_tiles ? row_ptr(n + 1) : nullptr;
      const int j_s = u.begin + n * kRows + 32 * quad + lane;  // the list entry of this thread's softmax row
      const int id_s = list_block(args, u, j_s);
      // ---- unpack, region by region; a region is free when the previous
      // tile's O^T product has left it (the first tile's always are)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        uint32_t h[4][4];
        raw.unpack_region(m, h);
        if (n > 0 && ok) ok = wait_bar_warp(sm, &sm.free_[m], par ^ 1u, fw);
        if (ok) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(sm.tile + (16 * m + 4 * quarter + i) * kDgBytes + row_u * 16) =
                make_uint4(h[i][0], h[i][1], h[i][2], h[i][3]);
          warp_publish(&sm.full[m], lane);
        }
        if (n + 1 < n_tiles) raw.load_region(next, m, quarter);
      }
      {
        uint32_t h[2][4];
        unpack_rope(raw.rope, h);
        if (n > 0 && ok) ok = wait_bar_warp(sm, &sm.free_[4], par ^ 1u, fw);
        if (ok) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<uint4*>(sm.tile + (kLatent / 8 + 2 * quarter + i) * kDgBytes + row_u * 16) =
                make_uint4(h[i][0], h[i][1], h[i][2], h[i][3]);
          warp_publish(&sm.full[4], lane);
        }
        if (n + 1 < n_tiles) raw.load_rope(next, quarter);
      }
      if (ok) ok = wait_bar_warp(sm, &sm.s_full, par, fw);
      tcgen05_fence_after();

      // ---- softmax: this thread has one row of the tile for 16 columns
      float z[16];
      bool vis = false, nan_row = false, need = false;
      if (has_cols && ok) {
        uint32_t sr[16];
        tmem_ld16(tbase + lane_base + 16 * cq, sr);
        const int pos = list_pos(u, j_s);
        vis = id_s >= 0 && (!u.masked || (pos <= me && (pos < args.sinks || pos > me - args.window)));
        nan_row = isnan(__uint_as_float(sr[0]));
        need = nan_row;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          z[j] = vis ? __uint_as_float(sr[j]) * qscale[j] : -INFINITY;
          need |= z[j] > m_ref[j] + kLazyRaise;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] = -INFINITY;
      }
      if (!ok) atomicMin(&sm.abort_tile, n);
      // every unpack thread takes the same branch at every barrier: a failed
      // wait is recorded with its tile before that tile's barrier
      const bool raise = compute_any(need);
      if (*reinterpret_cast<volatile int*>(&sm.abort_tile) <= n) {
        aborted = true;
        break;
      }
      if (raise) {
        // A cached row that holds a NaN makes its whole row of S NaN.  Columns
        // that see it get NaN through P; for those that do not, 0 x NaN must
        // not reach O^T, so the row's values leave the tile.
        if (nan_row && cq == 0) {
#pragma unroll 1
          for (int dg = 0; dg < kLatent / 8; ++dg)
            *reinterpret_cast<uint4*>(sm.tile + dg * kDgBytes + (32 * quad + lane) * 16) = make_uint4(0, 0, 0, 0);
        }
        float mx[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) mx[j] = z[j];
        const float m = reduce_cols(mx, lane, [](float a, float b) { return fmaxf(a, b); });
        if ((lane & 1) == 0) sm.red[warp][lane >> 1] = m;
        named_bar_sync(1, kComputeThreads);
        if (threadIdx.x < kCols) {
          const int w0 = threadIdx.x >> 4 << 2, c = threadIdx.x & 15;
          const float m4 = fmaxf(fmaxf(sm.red[w0][c], sm.red[w0 + 1][c]), fmaxf(sm.red[w0 + 2][c], sm.red[w0 + 3][c]));
          const float old = sm.m_ref[threadIdx.x];
          float al = 1.f;
          if (m4 > old + kLazyRaise) {
            al = ex2(old - m4);  // 0 while the maximum is -inf
            sm.m_ref[threadIdx.x] = m4;
          }
          sm.alpha[threadIdx.x] = al;
        }
        named_bar_sync(1, kComputeThreads);
        bool rescale = false;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float al = sm.alpha[16 * cq + j];
          l_part[j] *= al;
          rescale |= al != 1.f;
        }
        // O^T of the previous tiles is complete: S of this one came after it
        if (rescale && n > 0 && has_cols) {
#pragma unroll 1
          for (int m2 = 0; m2 < 4; ++m2) {
            const uint32_t ta = tbase + lane_base + kOCol + kCols * m2 + 16 * cq;
            uint32_t o[16];
            tmem_ld16(ta, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * sm.alpha[16 * cq + j]);
            tmem_st16(ta, o);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
      }
      if (has_cols) {
        uint32_t pk[8];
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          // The denominator sums P before its rounding to f16 (operand type of
          // the product): the LSE keeps float accuracy, and the output's share
          // of that rounding is at most 2^-11.
          const float p0 = vis ? ex2(z[j] - m_ref[j]) : 0.f;
          const float p1 = vis ? ex2(z[j + 1] - m_ref[j + 1]) : 0.f;
          l_part[j] += p0;
          l_part[j + 1] += p1;
          const __half2 ph = __floats2half2_rn(p0, p1);
          pk[j >> 1] = *reinterpret_cast<const uint32_t*>(&ph);
        }
#pragma unroll
        for (int g = 0; g < 2; ++g)
          *reinterpret_cast<uint4*>(sm.tile + kPOff + (2 * cq + g) * kDgBytes + (32 * quad + lane) * 16) =
              make_uint4(pk[4 * g], pk[4 * g + 1], pk[4 * g + 2], pk[4 * g + 3]);
      }
      tcgen05_fence_before();
      warp_publish(&sm.p_full, lane);
    }
    const bool ok = !aborted && wait_bar_warp(sm, &sm.done, 0u, fw);
    if (!compute_any(!ok)) {
      tcgen05_fence_after();
      const float l = reduce_cols(l_part, lane, [](float a, float b) { return a + b; });
      if ((lane & 1) == 0) sm.red[warp][lane >> 1] = l;
      named_bar_sync(1, kComputeThreads);
      if (threadIdx.x < u.ncols) {
        const int w0 = threadIdx.x >> 4 << 2, c = threadIdx.x & 15;
        const float lt = (sm.red[w0][c] + sm.red[w0 + 1][c]) + (sm.red[w0 + 2][c] + sm.red[w0 + 3][c]);
        sm.alpha[threadIdx.x] = lt == 0.f ? 0.f : 1.f / lt;  // 0 when the column saw nothing
        const float lse2 = lt == 0.f ? -INFINITY : sm.m_ref[threadIdx.x] + lg2(lt);
        if (!direct)
          args.part_lse[(u.col0 + threadIdx.x) * args.parts + u.part] = lse2;
        else if (args.lse != nullptr)
          args.lse[u.col0 + threadIdx.x] = lse2 * kLn2f;
      }
      named_bar_sync(1, kComputeThreads);
      if (has_cols) {
#pragma unroll 1
        for (int m = 0; m < 4; ++m) {
          uint32_t o[16];
          tmem_ld16(tbase + lane_base + kOCol + kCols * m + 16 * cq, o);
          const int dim = 128 * m + 32 * quad + lane;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float inv = sm.alpha[16 * cq + j];
            const float x = inv == 0.f ? 0.f : __uint_as_float(o[j]) * inv;
            const int64_t col = u.col0 + 16 * cq + j;
            if (direct)
              args.out[col * kLatent + dim] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
            else  // a convex combination of cached values (|x| <= 6 x 448): f16 keeps 11 significant bits
              args.part_o[(col * args.parts + u.part) * kLatent + dim] = __float2half_rn(x);
          }
        }
      }
    }
  }

  // ---- teardown: no MMA may be in flight when the CTA frees its tensor memory
  if (warp == kWarps && lane == 0) mbar_wait_bounded(&sm.done, 0u, fw, kFaultDecodeWait);
  tcgen05_fence_before();
  __syncthreads();
  if (warp == kWarps) {
    tcgen05_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(kTmemCols) : "memory");
  }
}

// Joins a column's partials: LSE = log2 sum 2^lse_s, out = sum 2^(lse_s - LSE)
// O_s.  One CTA per column, four dims per thread; the loads of a chunk of
// partials are all issued before the first is used.  A partial whose LSE is
// -inf was not written and is not read.
constexpr int kMergeChunk = 8;
__global__ void __launch_bounds__(128) dense_merge_kernel(const __half* __restrict__ part_o,
                                                          const float* __restrict__ part_lse, int parts,
                                                          uint16_t* __restrict__ out, float* __restrict__ lse) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t col = blockIdx.x;
  const int t = threadIdx.x;
  const float* pl = part_lse + col * parts;
  const uint2* src = reinterpret_cast<const uint2*>(part_o + col * parts * kLatent) + t;
  float mx = -INFINITY, wsum = 0.f;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < parts; s0 += kMergeChunk) {
    float ls[kMergeChunk];
    uint2 v[kMergeChunk];
#pragma unroll
    for (int i = 0; i < kMergeChunk; ++i) ls[i] = s0 + i < parts ? __ldg(pl + s0 + i) : -INFINITY;
#pragma unroll
    for (int i = 0; i < kMergeChunk; ++i)
      v[i] = ls[i] != -INFINITY ? __ldg(src + static_cast<int64_t>(s0 + i) * (kLatent / 4)) : make_uint2(0, 0);
    float cm = mx;
#pragma unroll
    for (int i = 0; i < kMergeChunk; ++i) cm = ls[i] > cm || isnan(ls[i]) ? ls[i] : cm;
    if (cm == -INFINITY) continue;  // nothing seen so far
    const float al = ex2(mx - cm);  // 0 while mx is -inf
    wsum *= al;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] *= al;
    mx = cm;
#pragma unroll
    for (int i = 0; i < kMergeChunk; ++i) {
      const float w = ex2(ls[i] - mx);
      wsum += w;
      const __half2 a = *reinterpret_cast<const __half2*>(&v[i].x), b = *reinterpret_cast<const __half2*>(&v[i].y);
      acc[0] += w * __low2float(a);
      acc[1] += w * __high2float(a);
      acc[2] += w * __low2float(b);
      acc[3] += w * __high2float(b);
    }
  }
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[2] * inv, acc[3] * inv);
  *reinterpret_cast<uint2*>(out + col * kLatent + 4 * t) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (lse != nullptr && t == 0) lse[col] = wsum == 0.f ? -INFINITY : (mx + lg2(wsum)) * kLn2f;
}

cudaError_t launch_dependent(const void* kernel, unsigned grid, unsigned block, size_t smem, void** params,
                             cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, params);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// How the rows are split: modelled time of one CTA = its tiles + kStartTiles
// (start-up, query load and output, in tiles), of the call = full waves of
// the prefix's CTAs, with the own rows' CTAs (no longer than the prefix's) in
// the SMs that the last of those waves leaves idle and in waves of their own
// after it, + the joining of the partials (about a tile, and a third of one
// for every 8).  In eighths of a tile; the fewest partials among equals.
DensePlan plan_dense_decode(int batch, int q_len, int num_heads, int64_t own_rows, int prefix_len) {
  constexpr int64_t kStartTiles = 3;
  DensePlan p{1, 1, 0, 0, 0};
  const int64_t sms = device_sm_count();
  const int64_t req_cols = static_cast<int64_t>(q_len) * num_heads;
  const int64_t columns = batch * req_cols;
  p.groups_per_req = static_cast<int>((req_cols + kCols - 1) / kCols);
  const int64_t own_groups = static_cast<int64_t>(batch) * p.groups_per_req;
  const int64_t own_tiles = own_rows > kRows ? (own_rows + kRows - 1) / kRows : 1;
  const int64_t pre_tiles = (static_cast<int64_t>(prefix_len) + kRows - 1) / kRows;
  const int64_t pre_groups = pre_tiles > 0 ? (columns + kCols - 1) / kCols : 0;
  p.prefix_groups = static_cast<int>(pre_groups);
  const int64_t tiles = pre_tiles > 0 ? pre_tiles : own_tiles;
  const int64_t groups = pre_tiles > 0 ? pre_groups : own_groups;
  int64_t best = -1;
  for (int64_t n = 1; n <= tiles && n <= sms; ++n) {
    const int64_t slice = (tiles + n - 1) / n;
    const int64_t waves = (groups * n + sms - 1) / sms;
    int64_t cost = 8 * waves * (slice + kStartTiles), s = 0;
    if (pre_tiles > 0) {
      const int64_t own_slice = own_tiles < slice ? own_tiles : slice;
      s = (own_tiles + own_slice - 1) / own_slice;
      const int64_t fit = (waves * sms - groups * n) * ((slice + kStartTiles) / (own_slice + kStartTiles));
      if (own_groups * s > fit) cost += 8 * ((own_groups * s - fit + sms - 1) / sms) * (own_slice + kStartTiles);
    }
    if (n + s > 1) cost += 8 + (n + s) / 3;
    if (best < 0 || cost < best) {
      best = cost;
      p.prefix_splits = static_cast<int>(pre_tiles > 0 ? n : 0);
      p.splits = static_cast<int>(pre_tiles > 0 ? s : n);
    }
    if (groups * n > 4 * sms) break;  // every SM has several CTAs already
  }
  const size_t parts = static_cast<size_t>(p.prefix_splits) + p.splits;
  if (parts > 1)
    p.workspace = (static_cast<size_t>(columns) * parts * (kLatent * sizeof(__half) + sizeof(float)) + 255) / 256 * 256;
  return p;
}

cudaError_t launch_dense_decode(int fmt, DenseArgs a, const DensePlan& plan, void* workspace, cudaStream_t stream) {
  a.groups_per_req = plan.groups_per_req;
  a.splits = plan.splits;
  a.prefix_groups = plan.prefix_groups;
  a.prefix_splits = plan.prefix_splits;
  a.parts = plan.prefix_splits + plan.splits;
  a.columns = static_cast<int64_t>(a.batch) * a.q_len * a.num_heads;
  a.fault_word = fault_word_ptr();
  if (a.fault_word == nullptr) return cudaErrorInvalidDevicePointer;
  if (a.parts > 1) {
    const size_t o_bytes = static_cast<size_t>(a.columns) * a.parts * kLatent * sizeof(__half);
    a.part_o = static_cast<__half*>(workspace);
    a.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + o_bytes);
  }
  const void* kernel = fmt == 0 ? reinterpret_cast<const void*>(dense_decode_kernel<0>)
                                : reinterpret_cast<const void*>(dense_decode_kernel<1>);
  static std::atomic<uint64_t> configured[2];
  cudaError_t e = set_smem_limit_once(kernel, static_cast<int>(sizeof(Smem)), &configured[fmt == 0 ? 0 : 1]);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(a.prefix_groups) * a.prefix_splits +
                        static_cast<int64_t>(a.batch) * a.groups_per_req * a.splits;
  void* params[] = {&a};
  e = launch_dependent(kernel, static_cast<unsigned>(units), kThreads, sizeof(Smem), params, stream);
  if (e != cudaSuccess || a.parts == 1) return e;
  const __half* po = a.part_o;
  const float* pl = a.part_lse;
  void* merge[] = {&po, &pl, &a.parts, &a.out, &a.lse};
  return launch_dependent(reinterpret_cast<const void*>(dense_merge_kernel), static_cast<unsigned>(a.columns), 128, 0,
                          merge, stream);
}

}  // namespace mla
