// Dense MLA decode over the paged cache on the fifth-generation tensor cores:
// a sliding window with first tokens that stay visible, and a batch whose
// requests share a prefix.  NVFP4 or FP8 rows, f16 operands, f32 accumulation.
//
// Mathematics.  64 "columns" -- (query token, head) pairs that look at the
// same cached rows -- share one walk over those rows, a cache block of 64 rows
// (one tile) at a time:
//   S[64 rows x 64 columns] = K[64 x 576] . Q^T
//   P = 2^(S scale - m), m the column's running maximum (raised lazily)
//   O^T[512 x 64] = O^T + V^T[512 x 64] . P,   V = the first 512 of K
// and each column's denominator is summed in float beside it, so the rows are
// read and unpacked once for all 64 columns.  A request's query tokens and
// heads fill columns; where the rows are a shared prefix, so do the requests.
//
// Work split.  One CTA = 64 columns x a slice of their blocks; slices' partial
// outputs (normalised, f16) and base-2 LSEs are joined by dense_merge_kernel.
// Roles: one lane issues every tcgen05.mma; one copies each block, which is
// contiguous, with one bulk copy into one of two slots; 8 warps unpack; 8 run
// the softmax; all 16 write the output.  The unpacked tile is stored once, as
// 8 x 8 core matrices, dim group major, which is at the same time the K-major A
// operand of S (M = 64 rows) and the MN-major A operand of O^T (M = 128 dims).
// It is handed over in five pieces (rope, 4 x 128 latent dims) through a ring
// that fills what shared memory the query and the block slots leave: two rope
// pieces and 4 (FP8, 64 columns) to 8 (NVFP4, 16 columns) latent ones.  A
// latent piece is refilled as soon as the O^T product has left it; with the
// pieces beyond a tile's own the next tile's unpacking and its part of S run
// during the softmax.  P lies in the tile's rope piece, which only S reads.
//
// Every wait is bounded; one that runs out sets the library's fault bit and
// the CTA leaves after its copies and MMAs in flight have drained.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kRows = kBlock;  // rows per tile: one cache block
constexpr int kCols = 64;      // columns per CTA
// Warp 0 issues the MMAs (a warp's instructions wait for those of older warps
// on its scheduler: as the youngest, it issued one MMA in ~200 cycles), warp 1
// copies, then the unpack and the softmax warps.
constexpr int kMmaWarp = 0;
constexpr int kCopyWarp = 1;
constexpr int kFirstUnpack = 2;
constexpr int kUnpackWarps = 8;
constexpr int kFirstSoftmax = kFirstUnpack + kUnpackWarps;
constexpr int kSoftmaxWarps = 8;
constexpr int kWarps = kUnpackWarps + kSoftmaxWarps;
constexpr int kComputeThreads = kWarps * 32;
constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
constexpr int kThreads = kComputeThreads + 32 * kFirstUnpack;
constexpr int kDimGroups = (kLatent + kRope) / 8;  // 72
// One 8-dim group of a tile: 16 bytes a row and 16 bytes of padding, see
// RawPiece.
constexpr int kDgBytes = kRows * 16 + 16;       // 1,040
constexpr int kLatPiece = 16 * kDgBytes;        // 128 latent dims: 16,640
constexpr int kRopePiece = 8 * kDgBytes;        // 64 rope dims, or P: 8,320
constexpr int kQGroupBytes = kDimGroups * 128;  // 8 columns x 576 dims: 9,216
constexpr int kMaxSlots = 2;
constexpr int kMaxPieces = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 128;  // S: columns 0-63 and 64-127 (tiles in turn), O^T: 128-383
// The maximum of a column is raised only when a score exceeds it by 2^8: P
// stays within 2^8 in f16 and O^T is rarely rescaled.
constexpr float kLazyRaise = 8.f;
constexpr int kPolls = 1 << 16;  // of the MMA warp, while it may do either of two things
constexpr float kLn2f = 0.6931471805599453f;

struct Ctl {               // the fixed part of shared memory, at its start
  float red[kSoftmaxWarps][32];  // per warp, per column reduction scratch
  float m_ref[kCols];      // running (lazy) maximum, base 2
  float alpha[kCols];      // factor of the last raise; at the end 1 / denominator
  float qscale[kCols];     // softmax scale (base 2) x 2^-shift of the column's query
  uint32_t qmax[kCols];    // largest |q| of the column (bf16 magnitude bits)
  uint64_t raw_full[kMaxSlots], raw_free[kMaxSlots];
  uint64_t rope_full[2], rope_free[2], full[kMaxPieces], free_[kMaxPieces];
  uint64_t s_full, p_full, done;
  uint32_t tmem_base;
  int abort_flag;  // set by whoever ran out of polls; ends the others' waits
  int abort_tile;  // first tile whose barrier a softmax warp reached with a failed wait
};
constexpr int kCtlBytes = 4096;
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");
constexpr int kSmemBytes = 227 * 1024;
constexpr int row_bytes(int fmt) { return fmt == 0 ? kRowNvfp4 : kRowFp8; }
// Latent pieces that fit beside the rest for a CTA of `cols` columns, and block
// slots: two where that leaves a piece beyond a tile's own, else one.
__host__ __device__ constexpr int latent_pieces(int fmt, int cols, int slots) {
  const int left = kSmemBytes - kCtlBytes - slots * kRows * row_bytes(fmt) - cols / 8 * kQGroupBytes - 2 * kRopePiece;
  return left / kLatPiece < kMaxPieces ? left / kLatPiece : kMaxPieces;
}
__host__ __device__ constexpr int block_slots(int fmt, int cols) { return latent_pieces(fmt, cols, 2) > 4 ? 2 : 1; }
static_assert(latent_pieces(0, kCols, block_slots(0, kCols)) >= 4 && latent_pieces(1, kCols, block_slots(1, kCols)) >= 4,
              "a whole tile must fit");

// ---- tcgen05 operands ---------------------------------------------------------
// No-swizzle shared-memory descriptor, in two words: start and byte offset
// between core matrices along K; byte offset between them along M / N (all
// >> 4) and descriptor version 1.  A later start adds its distance >> 4 to the
// low word, so the issuing lane spends two additions per MMA (descriptors
// built anew for each made it, not the tensor core, the limit).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t k_stride) {
  return ((saddr >> 4) & 0x3FFFu) | ((k_stride >> 4) << 16);
}
constexpr uint32_t desc_hi(uint32_t mn_stride) { return (mn_stride >> 4) | (1u << 14); }
// kind::f16, f16 operands, f32 accumulator; majorness 1 = MN-major.
__device__ __forceinline__ uint32_t f16_idesc(int m, int n, uint32_t a_mn, uint32_t b_mn) {
  return (1u << 4) | (a_mn << 15) | (b_mn << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}
template <uint32_t kAHi, uint32_t kBHi>
__device__ __forceinline__ void umma_f16(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 a, b; setp.ne.b32 p, %4, 0; mov.b64 a, {%1, %5}; mov.b64 b, {%2, %6}; "
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p; }" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "n"(kAHi), "n"(kBHi)
      : "memory");
}
// True in one lane of the (whole) warp.  MMAs behind this test issue every ~40
// cycles at N = 16 and ~48 at N = 64; behind `lane == 0` 45-50, predicated per
// MMA 66 (79 beside the unpack warps' stores).
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
  return e != 0;
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
// 16 lanes x 32 columns of this warp's quadrant (an M = 64 accumulator's rows
// 16 quad .. 16 quad + 15) in the matrix-fragment layout: r[4 k + e] is row
// lane / 4 + 8 (e / 2), column 8 k + 2 (lane % 4) + e % 2.
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// OR of `pred` over the softmax warps (named barrier 2).
__device__ __forceinline__ bool softmax_any(bool pred) {
  uint32_t out;
  asm volatile(
      "{ .reg .pred pi, po; setp.ne.u32 pi, %1, 0; barrier.cta.red.or.pred po, 2, %2, pi; selp.u32 %0, 1, 0, po; }"
      : "=r"(out)
      : "r"(static_cast<uint32_t>(pred)), "r"(kSoftmaxThreads)
      : "memory");
  return out != 0;
}
// Bounded wait for a phase.  The roles' loops share the instruction cache, so
// what follows the first poll stays out of line.
__device__ __noinline__ bool wait_bar_slow(int* abort_flag, uint64_t* bar, uint32_t parity, unsigned int* fw) {
  if (mbar_wait_or_abort(bar, parity, abort_flag, fw, kFaultDecodeWait)) return true;
  *reinterpret_cast<volatile int*>(abort_flag) = 1;
  return false;
}
__device__ __forceinline__ bool wait_bar(int* abort_flag, uint64_t* bar, uint32_t parity, unsigned int* fw) {
  return mbar_try_wait(bar, parity) || mbar_try_wait(bar, parity) || wait_bar_slow(abort_flag, bar, parity, fw);
}
__device__ __forceinline__ bool test_bar(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// The same for a whole warp: one lane polls.
__device__ __forceinline__ bool wait_bar_warp(int* abort_flag, uint64_t* bar, uint32_t parity, unsigned int* fw) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = wait_bar(abort_flag, bar, parity, fw);
  return __shfl_sync(0xFFFFFFFFu, static_cast<int>(ok), 0) != 0;
}
// One arrival per warp after all its lanes' shared-memory writes: each lane
// publishes its own writes to the tensor core's proxy first.
__device__ __forceinline__ void warp_publish(uint64_t* bar, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// How an unpack warp reads and writes its 8 rows.  The four lanes of a row hold
// its "quarters": 32 dims of each 128-dim region and 16 rope dims.  Eight
// lanes (one 16-byte shared-memory access) are two rows, r and r + 2.  Rows are
// 22 (NVFP4) or 36 (FP8) 16-byte pieces apart: the eight pieces read, 6 r + q
// (mod 8), fall into different banks; of FP8's two pieces a quarter, row r + 2
// reads the second first, 4 r + 2 q + h.  Stores go to dim groups 1,040 bytes
// apart; with quarters 2 and 3 one dim group ahead of 0 and 1, the pieces
// 4 q + (i + q / 2) % 4 + r (mod 8) differ as well.  Dim group i of a quarter is
// therefore given as its (i - q / 2)-th, and `ahead` is q / 2; `second` is row r + 2.
template <int FMT>
struct RawPiece;
template <>
struct RawPiece<0> {
  uint4 c;
  uint32_t two;  // the two scales
  __device__ __forceinline__ void load(const uint8_t* row, int m, int quarter, bool) {
    c = *reinterpret_cast<const uint4*>(row + 64 * m + 16 * quarter);
    two = *reinterpret_cast<const unsigned short*>(row + kScaleOff + 8 * m + 2 * quarter);
  }
  __device__ __forceinline__ void unpack(bool ahead, bool, uint32_t (&h)[4][4]) const {
    const uint32_t s0 = e4m3x2_to_f16x2((two & 0xFFu) * 0x0101u), s1 = e4m3x2_to_f16x2((two >> 8) * 0x0101u);
    const uint32_t w[4] = {ahead ? c.y : c.x, ahead ? c.z : c.y, ahead ? c.w : c.z, ahead ? c.x : c.w};
    const uint32_t s[4] = {s0, ahead ? s1 : s0, s1, ahead ? s0 : s1};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e2m1x8_to_f16x2x4(w[i], h[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) h[i][k] = hmul2(h[i][k], s[i]);
    }
  }
};
template <>
struct RawPiece<1> {
  uint4 x, y;
  __device__ __forceinline__ void load(const uint8_t* row, int m, int quarter, bool second) {
    const uint8_t* p = row + 128 * m + 32 * quarter;
    x = *reinterpret_cast<const uint4*>(p + (second ? 16 : 0));
    y = *reinterpret_cast<const uint4*>(p + (second ? 0 : 16));
  }
  __device__ __forceinline__ void unpack(bool ahead, bool second, uint32_t (&h)[4][4]) const {
    const uint4 c0 = second ? y : x, c1 = second ? x : y;
    const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo[2], hi[2];
      e4m3x4_to_f16x2x2(ahead ? w[(2 * i + 2) & 7] : w[2 * i], lo);
      e4m3x4_to_f16x2x2(ahead ? w[(2 * i + 3) & 7] : w[2 * i + 1], hi);
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

// One CTA's work: columns [col0, col0 + ncols) over tiles [begin, end) of a
// list of cache blocks.  Tile t is logical block t for t < n_sink_blocks, else
// w_block + t - n_sink_blocks.  Positions in [0, stop) that lie in the first
// `sinks` or from w0 on are seen by some column.
struct Unit {
  int64_t col0;
  int ncols;
  int part;  // slot of its partial among a column's
  const int32_t* table;
  int table_len;
  int n_sink_blocks, w_block, begin, end;
  int sinks, w0, stop;
  int tok_col0;  // col0 within its request (own rows)
  int me0;       // position of query token 0 (own rows)
  bool masked;   // own rows: visibility depends on the query token
};

__device__ __forceinline__ Unit find_unit(const DenseArgs& a) {
  Unit u;
  const int id = blockIdx.x;
  const int n_prefix = a.prefix_groups * a.prefix_splits;
  int sp, splits;
  u.tok_col0 = u.me0 = 0;
  if (id < n_prefix) {
    sp = id % a.prefix_splits;
    splits = a.prefix_splits;
    u.col0 = static_cast<int64_t>(id / a.prefix_splits) * kCols;
    u.ncols = static_cast<int>(min(static_cast<int64_t>(kCols), a.columns - u.col0));
    u.part = sp;
    u.table = a.prefix_table;
    u.table_len = (a.prefix_len + kBlock - 1) / kBlock;
    u.sinks = 0;
    u.w0 = 0;
    u.stop = a.prefix_len;
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
    u.stop = max(0, static_cast<int>(min(static_cast<int64_t>(me_hi) + 1, held)));
    u.sinks = min(a.sinks, u.stop);
    u.w0 = max(u.sinks, me_lo - a.window + 1);
  }
  u.n_sink_blocks = (u.sinks + kBlock - 1) / kBlock;
  u.w_block = max(u.w0 / kBlock, u.n_sink_blocks);
  const int tiles = u.n_sink_blocks + max(0, (u.stop + kBlock - 1) / kBlock - u.w_block);
  // spread evenly over the splits
  u.begin = static_cast<int>(static_cast<int64_t>(tiles) * sp / splits);
  u.end = static_cast<int>(static_cast<int64_t>(tiles) * (sp + 1) / splits);
  return u;
}
__device__ __forceinline__ int tile_block(const Unit& u, int t) {
  return t < u.n_sink_blocks ? t : u.w_block + (t - u.n_sink_blocks);
}
// Physical block of tile t as the table has it (it may lie outside the pool),
// -1 past the slice or the table.
__device__ __forceinline__ int tile_id(const Unit& u, int t) {
  if (t >= u.end) return -1;
  const int blk = tile_block(u, t);
  return blk < u.table_len ? __ldg(u.table + blk) : -1;
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) dense_decode_kernel(const DenseArgs args) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Ctl& sm = *reinterpret_cast<Ctl*>(smem_raw);
  constexpr int kRowBytes = row_bytes(FMT);
  constexpr uint32_t kBlockBytes = kRows * kRowBytes;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cw = warp - kFirstUnpack, ct = threadIdx.x - 32 * kFirstUnpack;  // among the unpack and softmax warps
  unsigned int* fw = args.fault_word;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Unit u = find_unit(args);
  const int n_tiles = u.end - u.begin;
  const int n_slots = block_slots(FMT, u.ncols);
  const int n_pieces = latent_pieces(FMT, u.ncols, n_slots);
  uint8_t* const s_raw = smem_raw + kCtlBytes;                  // blocks as stored
  uint8_t* const s_q = s_raw + n_slots * kBlockBytes;           // (col / 8) * 9216 + (dim / 8) * 128 + (col % 8) * 16
  uint8_t* const s_rope = s_q + u.ncols / 8 * kQGroupBytes;     // (dim / 8) * 1040 + row * 16 + (dim % 8) * 2
  uint8_t* const s_lat = s_rope + 2 * kRopePiece;               // likewise, 128 dims a piece
  const bool direct = args.parts == 1;
  const unsigned pool_blocks = static_cast<unsigned>(min(args.num_blocks, static_cast<int64_t>(0x7FFFFFFF)));
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
  if (warp >= kFirstUnpack && ct < kCols) {
    sm.m_ref[ct] = -INFINITY;
    sm.qmax[ct] = 0;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(&sm.raw_full[i], 1);
      mbar_init(&sm.raw_free[i], kUnpackWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.rope_full[i], kUnpackWarps);
      mbar_init(&sm.rope_free[i], 1);
    }
    for (int i = 0; i < kMaxPieces; ++i) {
      mbar_init(&sm.full[i], kUnpackWarps);
      mbar_init(&sm.free_[i], 1);
    }
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.p_full, kSoftmaxWarps);
    mbar_init(&sm.done, 1);
    sm.abort_flag = 0;
    sm.abort_tile = 0x7FFFFFFF;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  constexpr uint32_t tbase = 0;  // all 512 columns were allocated: they start at column 0
  int copied = 0;  // copying lane: tiles whose copy it has started

  // The copy of tile n, once its slot is free: one contiguous block, or none
  // where the table names no block of the pool.
  auto copy_tile = [&](int n, int id) {
    const int slot = n % n_slots;
    if (n >= n_slots && !wait_bar(&sm.abort_flag, &sm.raw_free[slot], static_cast<uint32_t>(n / n_slots - 1) & 1u, fw))
      return false;
    if (static_cast<unsigned>(id) < pool_blocks) {
      mbar_expect_tx(&sm.raw_full[slot], kBlockBytes);
      bulk_load(s_raw + slot * kBlockBytes, args.pool + static_cast<int64_t>(id) * args.block_stride, kBlockBytes,
                &sm.raw_full[slot]);
    } else {
      mbar_arrive(&sm.raw_full[slot]);
    }
    copied = n + 1;
    return true;
  };
  if (warp == kCopyWarp && lane == 0) {  // the first blocks arrive while the query is converted
    for (int n = 0; n < n_slots && n < n_tiles; ++n) copy_tile(n, tile_id(u, u.begin + n));
  }
  if (warp >= kFirstUnpack) {
    // The query, bf16 -> f16 core matrices of 8 columns x 8 dims.  A warp moves
    // 8 columns x 32 dims at a time (64-byte pieces of 8 rows in, conflict-free
    // 16-byte stores out); every load is issued before the first is used.  A
    // column whose query holds an infinity or NaN enters as zeros with a NaN
    // scale: its results are NaN, its neighbours' are not.
    constexpr int kPieces = kDimGroups / 4;               // of 32 dims
    constexpr int kPer = (kCols / 8) * kPieces / kWarps;  // 9
    const int n_tasks = (u.ncols / 8) * kPieces;
    uint4 x[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int task = cw + i * kWarps;
      const int64_t col = u.col0 + task / kPieces * 8 + (lane & 7);
      const int dg = task % kPieces * 4 + (lane >> 3);
      x[i] = make_uint4(0, 0, 0, 0);
      if (task < n_tasks)
        x[i] = dg < kLatent / 8
                   ? __ldg(reinterpret_cast<const uint4*>(args.q_nope + col * kLatent) + dg)
                   : __ldg(reinterpret_cast<const uint4*>(args.q_rope + col * kRope) + (dg - kLatent / 8));
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int task = cw + i * kWarps;
      if (task >= n_tasks) break;
      uint32_t mx = bf16x8_absmax_bits(x[i]);
      mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
      mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
      if (lane < 8) atomicMax(&sm.qmax[task / kPieces * 8 + lane], mx);
    }
    named_bar_sync(1, kComputeThreads);
    if (ct < kCols) {
      const uint32_t mx = sm.qmax[ct];
      sm.qscale[ct] = mx >= 0x7F80u ? __int_as_float(0x7FFFFFFF) : args.scale_log2 * pow2f(-query_shift(mx));
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int task = cw + i * kWarps;
      if (task >= n_tasks) break;
      const int hg = task / kPieces;
      const int dg = task % kPieces * 4 + (lane >> 3);
      const uint32_t mx = sm.qmax[hg * 8 + (lane & 7)];
      const float mul = pow2f(query_shift(mx));
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        h[k] = mx >= 0x7F80u ? 0u
                             : f32x2_to_f16x2_sat(bf16_bits_to_f32(w[k] & 0xFFFFu) * mul,
                                                  bf16_bits_to_f32(w[k] >> 16) * mul);
      *reinterpret_cast<uint4*>(s_q + hg * kQGroupBytes + dg * 128 + (lane & 7) * 16) =
          make_uint4(h[0], h[1], h[2], h[3]);
    }
    fence_proxy_async_smem();
  }
  __syncthreads();

  if (warp == kCopyWarp) {
    // ------------------------------------------------------------ copies
    if (lane == 0) {
      int id = tile_id(u, u.begin + n_slots);
      for (int n = n_slots; n < n_tiles; ++n) {
        const int next = tile_id(u, u.begin + n + 1);  // in flight while the slot is waited for
        if (!copy_tile(n, id)) break;
        id = next;
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    // One lane runs the whole role: an MMA piece of 8 then issues in ~190 cycles
    // (N = 16) to ~260 (N = 64), the tensor core's own rate; a warp-wide loop
    // with the MMAs behind an election in each turn took 370-410, and rolled
    // loops, whose operand registers wait for the previous MMA to start, ~800.
    const uint32_t idesc_s = f16_idesc(64, u.ncols, 0, 0);
    const uint32_t idesc_o = f16_idesc(128, u.ncols, 1, 1);
    const uint32_t rope0 = smem_u32(s_rope);
    const uint32_t q_b = desc_lo(smem_u32(s_q), 128);
    const uint32_t lat_s = desc_lo(rope0 + 2 * kRopePiece, kDgBytes), rope_s = desc_lo(rope0, kDgBytes);
    const uint32_t lat_o = desc_lo(rope0 + 2 * kRopePiece, 128), p_o = desc_lo(rope0, 128);
    if (elect_one()) {
      // Ring position of the next S piece and the next O^T piece, as slot, operand
      // address and (S) phase.
      int s_slot = 0, o_slot = 0;
      uint32_t s_a = lat_s, o_a = lat_o, s_phase = 0;
      bool ok = true;
#pragma unroll 1
      for (int n = -1; n < n_tiles && ok; ++n) {
        // S of tile n + 1 piece by piece -- rope (k = 0), then 128 latent dims each
        // (k = 1..4), 16 dims an MMA -- as its pieces fill, and O^T of tile n as
        // soon as its P is there.  The last piece of S comes after that: S is
        // complete only after O^T, so the softmax may rescale O^T, and P of two
        // tiles is never outstanding.
        const uint32_t next = static_cast<uint32_t>(n + 1), par = static_cast<uint32_t>(n) & 1u;
        const int k_end = n + 1 < n_tiles ? 5 : 0;
        const int k_early = min(k_end, min(4, 1 + n_pieces - 4));  // more cannot be there before O^T
        bool o_left = n >= 0;
        int k = 0, polls = 0;
        uint32_t s_b = q_b;
#pragma unroll 1
        while (k < k_end || o_left) {
          uint64_t* const bar = k == 0 ? &sm.rope_full[next & 1] : &sm.full[s_slot];
          const uint32_t bar_par = k == 0 ? (next >> 1) & 1u : s_phase;
          if (o_left && test_bar(&sm.p_full, par)) {
            tcgen05_fence_after();
            // O^T += V^T . P, 128 dims at a time, 16 rows an MMA
            const uint32_t p = p_o + (n & 1) * (kRopePiece >> 4);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
#pragma unroll
              for (int j = 0; j < kRows / 16; ++j)
                umma_f16<desc_hi(kDgBytes), desc_hi(kDgBytes)>(kOCol + kCols * m, o_a + j * (256 >> 4),
                                                               p + j * (256 >> 4), idesc_o, n > 0 || j > 0);
              umma_commit(&sm.free_[o_slot]);
              if (m == 3) umma_commit(&sm.rope_free[n & 1]);  // P is free when all four are done
              o_a += kLatPiece >> 4;
              if (++o_slot == n_pieces) {
                o_slot = 0;
                o_a = lat_o;
              }
            }
            o_left = false;
            polls = 0;
          } else if (k < (o_left ? k_early : k_end) && test_bar(bar, bar_par)) {
            tcgen05_fence_after();
            const uint32_t d = kCols * (next & 1);
            if (k == 0) {
              const uint32_t a = rope_s + (next & 1) * (kRopePiece >> 4), b = q_b + kLatent / 8 * (128 >> 4);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                umma_f16<desc_hi(128), desc_hi(kQGroupBytes)>(d, a + 2 * i * (kDgBytes >> 4), b + 2 * i * (128 >> 4),
                                                              idesc_s, i != 0);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                umma_f16<desc_hi(128), desc_hi(kQGroupBytes)>(d, s_a + 2 * i * (kDgBytes >> 4),
                                                              s_b + 2 * i * (128 >> 4), idesc_s, true);
              if (k == 4) umma_commit(&sm.s_full);
              s_b += 16 * (128 >> 4);
              s_a += kLatPiece >> 4;
              if (++s_slot == n_pieces) {
                s_slot = 0;
                s_a = lat_s;
                s_phase ^= 1u;
              }
            }
            ++k;
            polls = 0;
          } else if (++polls == kPolls) {  // something is late: a bounded wait for what must come first
            ok = o_left ? wait_bar(&sm.abort_flag, &sm.p_full, par, fw) : wait_bar(&sm.abort_flag, bar, bar_par, fw);
            if (!ok) break;
            polls = 0;
          }
        }
      }
      umma_commit(&sm.done);  // arrives once every MMA issued above has completed
    }
    __syncwarp();
  } else if (warp < kFirstSoftmax) {
    // ------------------------------------------------------------ unpack
    const int quarter = lane & 3;
    const bool ahead = quarter >= 2, second = (lane & 4) != 0;
    const int row_u = 8 * cw + ((lane >> 3) & 1) + (lane >> 4) * 4 + (second ? 2 : 0);
    int id = tile_id(u, u.begin);
    int piece = 0;         // next latent piece of the ring
    uint32_t phase = 1;    // of its release: the first round finds every piece free
    bool ok = true;
    for (int n = 0; n < n_tiles && ok; ++n) {
      const int slot = n % n_slots;
      // rows that no column sees enter as zeros, whatever the memory holds
      const int pos = tile_block(u, u.begin + n) * kBlock + row_u;
      const bool seen = static_cast<unsigned>(id) < pool_blocks && pos < u.stop && (pos < u.sinks || pos >= u.w0);
      id = tile_id(u, u.begin + n + 1);
      ok = wait_bar_warp(&sm.abort_flag, &sm.raw_full[slot], static_cast<uint32_t>(n / n_slots) & 1u, fw);
      if (!ok) break;
      const uint8_t* row = s_raw + slot * kBlockBytes + row_u * kRowBytes;
      RawPiece<FMT> raw;
      {
        uint32_t h[2][4];
        unpack_rope(*reinterpret_cast<const uint4*>(row + (FMT == 0 ? kRopeOffNvfp4 : kRopeOffFp8) + 16 * quarter), h);
        raw.load(row, 0, quarter, second);
        if (n >= 2)
          ok = wait_bar_warp(&sm.abort_flag, &sm.rope_free[n & 1], static_cast<uint32_t>((n >> 1) - 1) & 1u, fw);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<uint4*>(s_rope + (n & 1) * kRopePiece + (2 * quarter + i) * kDgBytes + row_u * 16) =
              seen ? make_uint4(h[i][0], h[i][1], h[i][2], h[i][3]) : make_uint4(0, 0, 0, 0);
      }
      // A piece is published only after the next one's conversion: its stores
      // have then long landed, which the proxy fence would wait for.
      uint64_t* stored = &sm.rope_full[n & 1];
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        uint32_t h[4][4];
        raw.unpack(ahead, second, h);
        warp_publish(stored, lane);
        if (m < 3) {
          raw.load(row, m + 1, quarter, second);
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.raw_free[slot]);  // every lane has read its last bytes of the block
        }
        ok = wait_bar_warp(&sm.abort_flag, &sm.free_[piece], phase, fw);
        if (!ok) break;
        uint8_t* dst = s_lat + piece * kLatPiece + 4 * quarter * kDgBytes + row_u * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(dst + ((i + (ahead ? 1 : 0)) & 3) * kDgBytes) =
              seen ? make_uint4(h[i][0], h[i][1], h[i][2], h[i][3]) : make_uint4(0, 0, 0, 0);
        stored = &sm.full[piece];
        if (++piece == n_pieces) {
          piece = 0;
          phase ^= 1u;
        }
      }
      if (ok) warp_publish(stored, lane);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int sw = warp - kFirstSoftmax;
    const int quad = warp & 3;        // tensor-memory lanes 32 quad .. 32 quad + 31
    const int half = sw >> 2;         // columns 32 half .. 32 half + 31
    const int c_lane = 2 * (lane & 3);
    const bool has_cols = 32 * half < u.ncols;
    const uint32_t lane_base = static_cast<uint32_t>(32 * quad) << 16;
    const int row0 = 16 * quad + (lane >> 2);  // this thread's rows: row0, row0 + 8
    float qs[8], mr[8];  // scale and maximum of columns 8 k + c_lane + e
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      qs[k] = sm.qscale[32 * half + 8 * (k >> 1) + c_lane + (k & 1)];
      mr[k] = -INFINITY;
    }
    // 16 columns share a query token
    const int me[2] = {u.me0 + (u.tok_col0 + 32 * half) / args.num_heads,
                       u.me0 + (u.tok_col0 + 32 * half + 16) / args.num_heads};
    float l_part[8];  // these rows' share of the denominators of columns 8 k + c_lane + e
#pragma unroll
    for (int j = 0; j < 8; ++j) l_part[j] = 0.f;
    int id = tile_id(u, u.begin);
    bool aborted = false;
    for (int n = 0; n < n_tiles; ++n) {
      const bool held = static_cast<unsigned>(id) < pool_blocks;
      id = tile_id(u, u.begin + n + 1);
      const int pos0 = tile_block(u, u.begin + n) * kBlock + row0;
      bool vis[2][2];  // [row][16-column half]
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int pos = pos0 + 8 * r;
          vis[r][c] = held && pos < u.stop &&
                      (!u.masked || (pos <= me[c] && (pos < args.sinks || pos > me[c] - args.window)));
        }
      bool ok = wait_bar_warp(&sm.abort_flag, &sm.s_full, static_cast<uint32_t>(n) & 1u, fw);
      tcgen05_fence_after();
      float z[16];
      bool nan_row[2] = {false, false}, need = false;
      if (has_cols && ok) {
        uint32_t sr[16];
        tmem_ld_rows16(tbase + lane_base + kCols * (n & 1) + 32 * half, sr);
#pragma unroll
        for (int r = 0; r < 2; ++r) nan_row[r] = isnan(__uint_as_float(sr[2 * r]));
        need = nan_row[0] || nan_row[1];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool on = 32 * half + 16 * (k >> 1) < u.ncols;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const bool v = on && vis[r][k >> 1];
            z[4 * k + 2 * r] = v ? __uint_as_float(sr[4 * k + 2 * r]) * qs[2 * k] : -INFINITY;
            z[4 * k + 2 * r + 1] = v ? __uint_as_float(sr[4 * k + 2 * r + 1]) * qs[2 * k + 1] : -INFINITY;
            need |= z[4 * k + 2 * r] > mr[2 * k] + kLazyRaise || z[4 * k + 2 * r + 1] > mr[2 * k + 1] + kLazyRaise;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] = -INFINITY;
      }
      if (!ok) atomicMin(&sm.abort_tile, n);
      // every softmax thread takes the same branch at every barrier: a failed
      // wait is recorded with its tile before that tile's barrier
      const bool raise = softmax_any(need);
      if (*reinterpret_cast<volatile int*>(&sm.abort_tile) <= n) {
        aborted = true;
        break;
      }
      if (raise) {
        // A cached row that holds a NaN makes its whole row of S NaN.  Columns
        // that see it get NaN through P; for those that do not, 0 x NaN must
        // not reach O^T, so the row's values leave the tile.
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (nan_row[r] && half == 0) {
#pragma unroll 1
            for (int dg = lane & 3; dg < kLatent / 8; dg += 4)
              *reinterpret_cast<uint4*>(s_lat + (4 * n + dg / 16) % n_pieces * kLatPiece + dg % 16 * kDgBytes +
                                        (row0 + 8 * r) * 16) = make_uint4(0, 0, 0, 0);
          }
        // maximum of each column: over this thread's two rows, the 8 lanes of
        // the column's pair, then the four warps of the half
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(z[4 * k + e], z[4 * k + 2 + e]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
            if (lane < 4) sm.red[4 * half + quad][8 * k + c_lane + e] = m;
          }
        named_bar_sync(3, kSoftmaxThreads);
        if (quad == 0) {
          const int c = 32 * half + lane;
          const float m4 = fmaxf(fmaxf(sm.red[4 * half][lane], sm.red[4 * half + 1][lane]),
                                 fmaxf(sm.red[4 * half + 2][lane], sm.red[4 * half + 3][lane]));
          const float old = sm.m_ref[c];
          float al = 1.f;
          if (m4 > old + kLazyRaise) {
            al = ex2(old - m4);  // 0 while the maximum is -inf
            sm.m_ref[c] = m4;
          }
          sm.alpha[c] = al;
        }
        named_bar_sync(3, kSoftmaxThreads);
        bool rescale = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 al = *reinterpret_cast<const float2*>(sm.alpha + 32 * half + 8 * k + c_lane);
          l_part[2 * k] *= al.x;
          l_part[2 * k + 1] *= al.y;
          rescale |= al.x != 1.f || al.y != 1.f;
          const float2 m = *reinterpret_cast<const float2*>(sm.m_ref + 32 * half + 8 * k + c_lane);
          mr[2 * k] = m.x;
          mr[2 * k + 1] = m.y;
        }
        // O^T of the previous tiles is complete: S of this one came after it
        if (n > 0 && has_cols && __any_sync(0xFFFFFFFFu, rescale)) {
#pragma unroll 1
          for (int m = 0; m < 8; ++m) {
            const uint32_t ta = tbase + lane_base + kOCol + kCols * (m >> 1) + 32 * half + 16 * (m & 1);
            uint32_t o[16];
            tmem_ld16(ta, o);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              o[j] = __float_as_uint(__uint_as_float(o[j]) * sm.alpha[32 * half + 16 * (m & 1) + j]);
            tmem_st16(ta, o);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
      }
      if (has_cols) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool on = 32 * half + 16 * (k >> 1) < u.ncols;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            // The denominator sums P before its rounding to f16 (operand type of
            // the product): the LSE keeps float accuracy, and the output's
            // share of that rounding is at most 2^-11.
            const bool v = on && vis[r][k >> 1];
            const float p0 = v ? ex2(z[4 * k + 2 * r] - mr[2 * k]) : 0.f;
            const float p1 = v ? ex2(z[4 * k + 2 * r + 1] - mr[2 * k + 1]) : 0.f;
            l_part[2 * k] += p0;
            l_part[2 * k + 1] += p1;
            const __half2 ph = __floats2half2_rn(p0, p1);
            *reinterpret_cast<__half2*>(s_rope + (n & 1) * kRopePiece + (4 * half + k) * kDgBytes +
                                        (row0 + 8 * r) * 16 + 2 * c_lane) = ph;
          }
        }
      }
      tcgen05_fence_before();
      warp_publish(&sm.p_full, lane);
    }
    // ---- denominators and LSEs, once every product is done
    const bool ok = !aborted && wait_bar_warp(&sm.abort_flag, &sm.done, 0u, fw);
    if (!ok) atomicMin(&sm.abort_tile, -1);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = l_part[2 * k + e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, off);
        if (lane < 4) sm.red[4 * half + quad][8 * k + c_lane + e] = l;
      }
    named_bar_sync(3, kSoftmaxThreads);
    if (quad == 0 && 32 * half + lane < u.ncols) {
      const int c = 32 * half + lane;
      const float lt = (sm.red[4 * half][lane] + sm.red[4 * half + 1][lane]) +
                       (sm.red[4 * half + 2][lane] + sm.red[4 * half + 3][lane]);
      sm.alpha[c] = lt == 0.f ? 0.f : 1.f / lt;  // 0 when the column saw nothing
      const float lse2 = lt == 0.f ? -INFINITY : sm.m_ref[c] + lg2(lt);
      if (*reinterpret_cast<volatile int*>(&sm.abort_tile) >= 0) {
        if (!direct)
          args.part_lse[(u.col0 + c) * args.parts + u.part] = lse2;
        else if (args.lse != nullptr)
          args.lse[u.col0 + c] = lse2 * kLn2f;
      }
    }
  }

  // ---- output: a warp has its quadrant's tensor-memory lanes and 16 columns
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  if (warp >= kFirstUnpack && 16 * (cw >> 2) < u.ncols && *reinterpret_cast<volatile int*>(&sm.abort_tile) >= 0) {
    const int quad = warp & 3, cq = cw >> 2;
#pragma unroll 1
    for (int m = 0; m < 4; ++m) {
      uint32_t o[16];
      tmem_ld16(tbase + (static_cast<uint32_t>(32 * quad) << 16) + kOCol + kCols * m + 16 * cq, o);
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

  // ---- teardown: no copy or MMA may be in flight when the CTA leaves or frees
  // its tensor memory
  if (warp == kCopyWarp && lane == 0) {
    for (int n = max(0, copied - n_slots); n < copied; ++n)
      mbar_wait_bounded(&sm.raw_full[n % n_slots], static_cast<uint32_t>(n / n_slots) & 1u, fw, kFaultDecodeWait);
  }
  if (warp == kMmaWarp && lane == 0) mbar_wait_bounded(&sm.done, 0u, fw, kFaultDecodeWait);
  tcgen05_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tcgen05_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sm.tmem_base), "r"(kTmemCols) : "memory");
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
// after it, + the joining of the partials (about two tiles, and one for every
// 12).  In eighths of a tile; the fewest partials among equals.
DensePlan plan_dense_decode(int batch, int q_len, int num_heads, int64_t own_rows, int prefix_len) {
  constexpr int64_t kStartTiles = 4;
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
    if (n + s > 1) cost += 16 + 2 * (n + s) / 3;
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
  cudaError_t e = set_smem_limit_once(kernel, kSmemBytes, &configured[fmt == 0 ? 0 : 1]);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(a.prefix_groups) * a.prefix_splits +
                        static_cast<int64_t>(a.batch) * a.groups_per_req * a.splits;
  void* params[] = {&a};
  e = launch_dependent(kernel, static_cast<unsigned>(units), kThreads, kSmemBytes, params, stream);
  if (e != cudaSuccess || a.parts == 1) return e;
  const __half* po = a.part_o;
  const float* pl = a.part_lse;
  void* merge[] = {&po, &pl, &a.parts, &a.out, &a.lse};
  return launch_dependent(reinterpret_cast<const void*>(dense_merge_kernel), static_cast<unsigned>(a.columns), 128, 0,
                          merge, stream);
}

}  // namespace mla
