// Dense MLA decode over the paged cache on the fifth-generation tensor cores:
// a sliding window with first tokens that stay visible, and a batch whose
// requests share a prefix.  NVFP4 or FP8 rows, f16 operands, f32 accumulation.
//
// Mathematics.  64 "columns" -- (query token, head) pairs that look at the
// same cached rows -- share one walk over those rows, half a cache block of 32
// rows (one tile) at a time:
//   S[64 columns x 32 rows] = Q[64 x 576] . K^T
//   P = 2^(S scale - r), r 9 below the column's running maximum (raised lazily)
//   O^T[512 x 64] = O^T + V^T[512 x 32] . P^T,   V = the first 512 of K
// and each column's denominator is summed in float beside it, so the rows are
// read and unpacked once for all 64 columns.  A request's query tokens and
// heads fill columns; where the rows are a shared prefix, so do the requests.
//
// Work split.  One CTA = 64 columns x a slice of their tiles; slices' partial
// outputs (normalised, float: behind a dominating row without a latent they can be
// far below f16's range) and base-2 LSEs are joined by dense_merge_kernel.
// Roles: one lane issues every tcgen05.mma; one copies each tile, which is
// contiguous, with one bulk copy; 8 warps unpack a tile (8 rows x half the dims
// each); 8 run its softmax (16 columns x 16 rows each); all write the output.
// The unpacked tile is stored once, as 8 x 8 core matrices, dim group major,
// which is at the same time the K-major B operand of S (N = 32 rows) and the
// MN-major A operand of O^T (M = 128 dims).  P lies in the tile's rope part,
// which only S reads.
//
// What bounds it.  The issuing lane: a tile takes it ~1,640 cycles, ~900 for the
// 36 MMAs of S (25 each, about what their operands take from shared memory), ~330
// for the 8 of O^T (41 each), ~270 for the two polls, which find what they ask for
// at the first or second try, ~150 for the two commits.  The tensor pipe is then
// active in half of the cycles.  The softmax's serial part is as long, so halving
// either alone changes nothing.  S of the next tile is issued before O^T of this
// one.  32 rows a tile and not 64 or 128, so that three unpacked tiles (37 KB each)
// fit beside a 72 KB query of 64 columns: pieces of 64-row tiles took 204 us where
// this took 118 (128 requests x 64 heads, window 4,096; 121 since P keeps far rows'
// weights), 64-row tiles beside 16 columns 68 to 81 us where this took 64 (32
// requests, window 8,192).  Slower as well: S two tiles ahead, an issuing lane for
// each product, two softmax sets on tiles in turn, and S of the next tile loaded
// while P is computed -- each delays O^T, which frees the tile.
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

constexpr int kRows = 32;  // rows per tile: half a cache block
constexpr int kCols = 64;  // columns per CTA
// Warp 0 issues the MMAs (a warp's instructions wait for those of older warps
// on its scheduler: as the youngest, it issued one MMA in ~200 cycles), warp 1
// copies, then the softmax and, as the youngest, the unpack warps.
constexpr int kMmaWarp = 0;
constexpr int kCopyWarp = 1;
constexpr int kFirstSoftmax = 2;
constexpr int kSoftmaxWarps = 8;  // two per tensor-memory quadrant: 16 columns x 16 rows of a tile each
constexpr int kFirstUnpack = kFirstSoftmax + kSoftmaxWarps;
constexpr int kUnpackWarps = 8;  // 8 rows x half the dims each
constexpr int kWarps = kUnpackWarps + kSoftmaxWarps;
constexpr int kComputeThreads = kWarps * 32;
constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
constexpr int kThreads = kComputeThreads + 32 * kFirstSoftmax;
constexpr int kDimGroups = (kLatent + kRope) / 8;  // 72
// One 8-dim group of a tile: 16 bytes a row and 16 bytes of padding, see
// RawPiece.
constexpr int kDgBytes = kRows * 16 + 16;             // 528
constexpr int kTileBytes = kDimGroups * kDgBytes;     // 38,016
constexpr int kPOff = kLatent / 8 * kDgBytes;         // P overlays the rope part
constexpr int kPGroupBytes = kRows / 8 * 128;         // P of 8 columns: 512
constexpr int kQGroupBytes = kDimGroups * 128;        // 8 columns x 576 dims: 9,216
constexpr int kMaxSlots = 4;                          // copied tiles
constexpr int kMaxTiles = 4;                          // unpacked tiles
static_assert(kCols / 8 * kPGroupBytes <= kRope / 8 * kDgBytes, "P fits the rope part");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 64;  // S: columns 0-31 and 32-63 (tiles in turn), O^T: 64-319
// P is f16, which has its full precision from 2^-14 to 2^16.  A raise puts a
// column's largest score so far at 2^9: a row keeps its weight to 2^-11 until it
// is 2^23 below the largest, and further down loses at most 2^-34 of the largest
// weight (with 10 instead of 9 2^24 and 2^-35, and 122.5 us where this takes 121:
// 128 requests x 64 heads, window 4,096, scores with a deviation of 3 bits).
// Scores that come later may reach 2^15.99 before the next raise, which, for
// whichever column it is, brings all 64 to their maxima: raising only the columns
// past the limit takes 155 us.
constexpr float kRaiseTo = 9.f;
constexpr float kRaiseAt = 15.99f;
constexpr float kLn2f = 0.6931471805599453f;

struct Ctl {              // the fixed part of shared memory, at its start
  float part[2][kCols];   // the row halves' maxima (at a raise) and denominators (at the end)
  float alpha[kCols];     // factor of the last raise; at the end 1 / denominator
  float qscale[kCols];    // softmax scale (base 2) x 2^-shift of the column's query
  uint32_t qmax[kCols];   // largest |q| of the column (bf16 magnitude bits)
  uint64_t raw_full[kMaxSlots], raw_free[kMaxSlots], full[kMaxTiles], free_[kMaxTiles];
  uint64_t s_full[2], p_full[2], done;
  uint32_t tmem_base;
  int abort_flag;  // set by whoever ran out of polls; ends the others' waits
  int abort_tile;  // first tile whose barrier a softmax warp reached with a failed wait
};
constexpr int kNoAbort = 0x7FFFFFFF;
constexpr int kCtlBytes = 2048;
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");
constexpr int kSmemBytes = 227 * 1024;
constexpr int row_bytes(int fmt) { return fmt == 0 ? kRowNvfp4 : kRowFp8; }
// Unpacked and copied tiles that fit beside the query of `cols` columns: first
// two copies, then unpacked tiles, then more copies.
__host__ __device__ constexpr int tile_room(int cols) { return kSmemBytes - kCtlBytes - cols / 8 * kQGroupBytes; }
__host__ __device__ constexpr int unpacked_tiles(int fmt, int cols) {
  const int n = (tile_room(cols) - 2 * kRows * row_bytes(fmt)) / kTileBytes;
  return n < kMaxTiles ? n : kMaxTiles;
}
__host__ __device__ constexpr int copied_tiles(int fmt, int cols) {
  const int n = (tile_room(cols) - unpacked_tiles(fmt, cols) * kTileBytes) / (kRows * row_bytes(fmt));
  return n < kMaxSlots ? n : kMaxSlots;
}
static_assert(unpacked_tiles(0, kCols) >= 3 && unpacked_tiles(1, kCols) >= 3, "three tiles in flight");

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
// 16 lanes x 16 columns of this warp's quadrant (rows 16 quad .. 16 quad + 15
// of an M = 64 accumulator) in the matrix-fragment layout: r[4 k + e] is row
// lane / 4 + 8 (e / 2), column 8 k + 2 (lane % 4) + e % 2.
__device__ __forceinline__ void tmem_ld_rows8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
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
// The same for a whole warp: every lane polls, and all go on or none.
__device__ __forceinline__ bool wait_bar_warp(int* abort_flag, uint64_t* bar, uint32_t parity, unsigned int* fw) {
  bool ok = true;
  if (!mbar_try_wait(bar, parity)) ok = wait_bar(abort_flag, bar, parity, fw);
  return __all_sync(0xFFFFFFFFu, ok);
}
// One arrival per warp after all its lanes' shared-memory writes: each lane
// publishes its own writes to the tensor core's proxy first.
__device__ __forceinline__ void warp_publish(uint64_t* bar, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// How an unpack warp reads and writes its 8 rows.  The four lanes of a row hold
// its "quarters": 32 dims of each 128-dim piece and 16 rope dims.  Eight lanes
// (one 16-byte shared-memory access) are two rows, r and r + 2.  Rows are 22
// (NVFP4) or 36 (FP8) 16-byte units apart: the eight units read, 6 r + q (mod
// 8), fall into different banks; of FP8's two units a quarter, row r + 2 reads
// the second first, 4 r + 2 q + h.  Stores go to dim groups 528 bytes apart;
// with quarters 2 and 3 one dim group ahead of 0 and 1, the units 4 q + (i + q /
// 2) % 4 + r (mod 8) differ as well.  Dim group i of a quarter is therefore
// given as its (i - q / 2)-th, and `ahead` is q / 2; `second` is row r + 2.
template <int FMT>
struct RawPiece;
template <>
struct RawPiece<0> {
  uint4 c;
  uint32_t two;  // the two scales
  __device__ __forceinline__ void load(const uint8_t* row, int m, int quarter, bool, bool seen) {
    c = *reinterpret_cast<const uint4*>(row + 64 * m + 16 * quarter);
    two = *reinterpret_cast<const unsigned short*>(row + kScaleOff + 8 * m + 2 * quarter);
    if (!seen) {
      c = make_uint4(0, 0, 0, 0);
      two = 0;
    }
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
  __device__ __forceinline__ void load(const uint8_t* row, int m, int quarter, bool second, bool seen) {
    const uint8_t* p = row + 128 * m + 32 * quarter;
    x = *reinterpret_cast<const uint4*>(p + (second ? 16 : 0));
    y = *reinterpret_cast<const uint4*>(p + (second ? 0 : 16));
    if (!seen) x = y = make_uint4(0, 0, 0, 0);
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
// One CTA's work: columns [col0, col0 + ncols) over tiles [begin, end) of a
// list.  Tile t is the t-th 32 positions for t < n_sink_tiles, else the (w_tile
// + t - n_sink_tiles)-th.  Positions in [0, stop) that lie in the first
// `sinks` or from w0 on are seen by some column.
struct Unit {
  int64_t col0;
  int ncols;
  int part;  // slot of its partial among a column's
  const int32_t* table;
  int table_len;
  int n_sink_tiles, w_tile, begin, end;
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
    const int ctx = min(max(a.ctx_lens[b], 0), a.max_context);
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
  u.n_sink_tiles = (u.sinks + kRows - 1) / kRows;
  u.w_tile = max(u.w0 / kRows, u.n_sink_tiles);
  const int tiles = u.n_sink_tiles + max(0, (u.stop + kRows - 1) / kRows - u.w_tile);
  // spread evenly over the splits
  u.begin = static_cast<int>(static_cast<int64_t>(tiles) * sp / splits);
  u.end = static_cast<int>(static_cast<int64_t>(tiles) * (sp + 1) / splits);
  return u;
}
// First position of tile t.
__device__ __forceinline__ int tile_pos(const Unit& u, int t) {
  return (t < u.n_sink_tiles ? t : u.w_tile + (t - u.n_sink_tiles)) * kRows;
}
// Physical block of tile t as the table has it (it may lie outside the pool),
// -1 past the slice or the table.  Lengths and tables are plain loads, which the
// wait for the kernel in front orders behind its writes: this grid may be resident
// before they are made, and the read-only path does not allow that.  (From L2, as
// the queries, they cost 2 %: 121 -> 123.5 us for 128 requests x 64 heads.)
__device__ __forceinline__ int tile_id(const Unit& u, int t) {
  if (t >= u.end) return -1;
  const int blk = tile_pos(u, t) / kBlock;
  return blk < u.table_len ? u.table[blk] : -1;
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) dense_decode_kernel(const DenseArgs args) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Ctl& sm = *reinterpret_cast<Ctl*>(smem_raw);
  constexpr int kRowBytes = row_bytes(FMT);
  constexpr uint32_t kRawBytes = kRows * kRowBytes;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cw = warp - kFirstSoftmax, ct = threadIdx.x - 32 * kFirstSoftmax;  // among the softmax and unpack warps
  unsigned int* fw = args.fault_word;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Unit u = find_unit(args);
  const int n_tiles = u.end - u.begin;
  const int n_slots = copied_tiles(FMT, u.ncols), n_bufs = unpacked_tiles(FMT, u.ncols);
  // The query comes first: S reads 64 columns of it, of which those past ncols
  // are whatever follows (rows of S that nobody uses).
  uint8_t* const s_q = smem_raw + kCtlBytes;                 // (col / 8) * 9216 + (dim / 8) * 128 + (col % 8) * 16
  uint8_t* const s_tile = s_q + u.ncols / 8 * kQGroupBytes;  // (dim / 8) * 528 + row * 16 + (dim % 8) * 2
  uint8_t* const s_raw = s_tile + n_bufs * kTileBytes;       // tiles as stored
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
  if (warp >= kFirstSoftmax && ct < kCols) sm.qmax[ct] = 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(&sm.raw_full[i], 1);
      mbar_init(&sm.raw_free[i], kUnpackWarps);
    }
    for (int i = 0; i < kMaxTiles; ++i) {
      mbar_init(&sm.full[i], kUnpackWarps);
      mbar_init(&sm.free_[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], kSoftmaxWarps);
    }
    mbar_init(&sm.done, 1);
    sm.abort_flag = 0;
    sm.abort_tile = kNoAbort;
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
  // all 512 tensor-memory columns were allocated: they start at column 0
  int copied = 0;  // copying lane: tiles whose copy it has started

  // The copy of tile n, once its slot is free: 32 contiguous rows, or none where
  // the table names no block of the pool.
  auto copy_tile = [&](int n, int id) {
    const int slot = n % n_slots;
    if (n >= n_slots && !wait_bar(&sm.abort_flag, &sm.raw_free[slot], static_cast<uint32_t>(n / n_slots - 1) & 1u, fw))
      return false;
    uint64_t* const full = &sm.raw_full[slot];
    if (static_cast<unsigned>(id) < pool_blocks) {
      mbar_expect_tx(full, kRawBytes);
      bulk_load(s_raw + slot * kRawBytes,
                args.pool + static_cast<int64_t>(id) * args.block_stride +
                    tile_pos(u, u.begin + n) % kBlock * kRowBytes,
                kRawBytes, full);
    } else {
      mbar_arrive(full);
    }
    copied = n + 1;
    return true;
  };
  if (warp == kCopyWarp && lane == 0) {  // the first tiles arrive while the query is converted
    for (int n = 0; n < n_slots && n < n_tiles; ++n) copy_tile(n, tile_id(u, u.begin + n));
  }
  if (warp >= kFirstSoftmax) {
    // The query, bf16 -> f16 core matrices of 8 columns x 8 dims.  A warp moves
    // 8 columns x 32 dims at a time (64-byte pieces of 8 rows in, conflict-free
    // 16-byte stores out); every load is issued before the first is used.  A
    // column whose query holds an infinity or NaN enters as zeros with a NaN
    // scale: its results are NaN, its neighbours' are not.  Coherent loads, as an
    // earlier call's output may be the query.
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
                   ? __ldcg(reinterpret_cast<const uint4*>(args.q_nope + col * kLatent) + dg)
                   : __ldcg(reinterpret_cast<const uint4*>(args.q_rope + col * kRope) + (dg - kLatent / 8));
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
    // One lane runs the whole role with a tile's MMAs unrolled: they then issue
    // at the tensor core's own rate (25 cycles at M = 64, N = 32; 41-48 at M =
    // 128).  A warp-wide loop with an election per piece took twice that, and
    // rolled loops, whose operand registers wait for the previous MMA to
    // start, four times.
    const uint32_t idesc_s = f16_idesc(64, kRows, 0, 0);
    const uint32_t idesc_o = f16_idesc(128, u.ncols, 1, 0);
    const uint32_t q_a = desc_lo(smem_u32(s_q), 128);
    const uint32_t tile_s = desc_lo(smem_u32(s_tile), kDgBytes), tile_o = desc_lo(smem_u32(s_tile), 128);
    const uint32_t tile_p = desc_lo(smem_u32(s_tile) + kPOff, 128);
    if (elect_one()) {
      int s_buf = 0, o_buf = 0;
      uint32_t s_phase = 0;
      bool ok = true;
#pragma unroll 1
      for (int n = 0; n <= n_tiles && ok; ++n) {
        if (n < n_tiles) {  // S of tile n, 16 dims an MMA
          ok = wait_bar(&sm.abort_flag, &sm.full[s_buf], s_phase, fw);
          if (!ok) break;
          tcgen05_fence_after();
          const uint32_t b = tile_s + s_buf * (kTileBytes >> 4), d = kRows * (n & 1);
#pragma unroll
          for (int i = 0; i < kDimGroups / 2; ++i)
            umma_f16<desc_hi(kQGroupBytes), desc_hi(128)>(d, q_a + 2 * i * (128 >> 4), b + 2 * i * (kDgBytes >> 4),
                                                          idesc_s, i != 0);
          umma_commit(&sm.s_full[n & 1]);
          if (++s_buf == n_bufs) {
            s_buf = 0;
            s_phase ^= 1u;
          }
        }
        if (n > 0) {  // O^T += V^T . P^T of tile n - 1, 128 dims at a time, 16 rows an MMA
          ok = wait_bar(&sm.abort_flag, &sm.p_full[(n - 1) & 1], static_cast<uint32_t>((n - 1) >> 1) & 1u, fw);
          if (!ok) break;
          tcgen05_fence_after();
          const uint32_t a = tile_o + o_buf * (kTileBytes >> 4), b = tile_p + o_buf * (kTileBytes >> 4);
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int i = 0; i < kRows / 16; ++i)
              umma_f16<desc_hi(kDgBytes), desc_hi(kPGroupBytes)>(kOCol + kCols * m,
                                                                 a + 16 * m * (kDgBytes >> 4) + i * (256 >> 4),
                                                                 b + i * (256 >> 4), idesc_o, n > 1 || i > 0);
          umma_commit(&sm.free_[o_buf]);
          if (++o_buf == n_bufs) o_buf = 0;
        }
      }
      umma_commit(&sm.done);  // arrives once every MMA issued above has completed
    }
    __syncwarp();
  } else if (warp >= kFirstUnpack) {
    // ------------------------------------------------------------ unpack
    const int uw = warp - kFirstUnpack;
    const int half = uw >> 2;  // dims 256 half .. 256 half + 255 and rope dims 32 half .. 32 half + 31
    const int quarter = lane & 3;
    const bool ahead = quarter >= 2, second = (lane & 4) != 0;
    const int row_u = 8 * (uw & 3) + ((lane >> 3) & 1) + (lane >> 4) * 4 + (second ? 2 : 0);
    int id = tile_id(u, u.begin);
    bool ok = true;
    int slot = 0, buf = 0;
    uint32_t full_phase = 0, free_phase = 1;
    for (int n = 0; n < n_tiles && ok; ++n) {
      // rows that no column sees enter as zeros, whatever the memory holds
      const int pos = tile_pos(u, u.begin + n) + row_u;
      const bool seen = static_cast<unsigned>(id) < pool_blocks && pos < u.stop && (pos < u.sinks || pos >= u.w0);
      id = tile_id(u, u.begin + n + 1);
      ok = wait_bar_warp(&sm.abort_flag, &sm.raw_full[slot], full_phase, fw);
      if (!ok) break;
      const uint8_t* row = s_raw + slot * kRawBytes + row_u * kRowBytes;
      uint8_t* dst = s_tile + buf * kTileBytes + row_u * 16;
      RawPiece<FMT> raw[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) raw[m].load(row, 2 * half + m, quarter, second, seen);
      uint2 rope = *reinterpret_cast<const uint2*>(row + (FMT == 0 ? kRopeOffNvfp4 : kRopeOffFp8) + 32 * half +
                                                   8 * quarter);
      if (!seen) rope = make_uint2(0, 0);
      // The copy has been read.  The next one writes the slot through another
      // proxy, so each lane's reads are fenced: without it they may still be on
      // their way, behind the tensor core's reads, when that copy lands.
      warp_publish(&sm.raw_free[slot], lane);
      if (n >= n_bufs) ok = wait_bar_warp(&sm.abort_flag, &sm.free_[buf], free_phase, fw);
      if (!ok) break;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t h[4][4];
        raw[m].unpack(ahead, second, h);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(dst + (32 * half + 16 * m + 4 * quarter + ((i + (ahead ? 1 : 0)) & 3)) * kDgBytes) =
              make_uint4(h[i][0], h[i][1], h[i][2], h[i][3]);
      }
      uint32_t lo[2], hi[2];
      e4m3x4_to_f16x2x2(rope.x, lo);
      e4m3x4_to_f16x2x2(rope.y, hi);
      *reinterpret_cast<uint4*>(dst + (kLatent / 8 + 4 * half + quarter) * kDgBytes) =
          make_uint4(lo[0], lo[1], hi[0], hi[1]);
      warp_publish(&sm.full[buf], lane);
      if (++slot == n_slots) {
        slot = 0;
        full_phase ^= 1u;
      }
      if (++buf == n_bufs) {
        buf = 0;
        free_phase ^= 1u;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int quad = warp & 3;          // tensor-memory lanes 32 quad ..: columns 16 quad .. 16 quad + 15
    const int rh = cw >> 2;             // rows 16 rh .. 16 rh + 15 of a tile
    const int t_lane = 2 * (lane & 3);  // of them, rows 8 k + t_lane + e
    const int col0 = 16 * quad + (lane >> 2);  // this thread's columns: col0, col0 + 8
    const bool has_cols = 16 * quad < u.ncols;
    const uint32_t lane_base = static_cast<uint32_t>(32 * quad) << 16;
    const int me = u.me0 + (u.tok_col0 + 16 * quad) / args.num_heads;  // 16 columns share a query token
    float qs[2] = {0.f, 0.f}, ref[2] = {-INFINITY, -INFINITY};  // scale and what P is relative to, base 2
    float top[2] = {-INFINITY, -INFINITY};                      // largest scores of this thread's rows so far
    float l_part[2] = {0.f, 0.f};  // these rows' share of the denominators
    if (has_cols) {
      qs[0] = sm.qscale[col0];
      qs[1] = sm.qscale[col0 + 8];
    }
    // bit 2 k + e: row 8 k + t_lane + e of this half of tile n, in block `id`, is seen
    auto seen_rows = [&](int n, int id) -> uint32_t {
      if (static_cast<unsigned>(id) >= pool_blocks) return 0;
      const int first = tile_pos(u, u.begin + n) + 16 * rh, last = first + 15;
      if (last < u.stop && (!u.masked || (last <= me && (last < args.sinks || first > me - args.window)))) return 15u;
      uint32_t v = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int pos = first + t_lane + 8 * (k >> 1) + (k & 1);
        if (pos < u.stop && (!u.masked || (pos <= me && (pos < args.sinks || pos > me - args.window)))) v |= 1u << k;
      }
      return v;
    };
    uint32_t vis = seen_rows(0, tile_id(u, u.begin));
    int id = tile_id(u, u.begin + 1);
    int buf = 0;
    bool aborted = false;
    for (int n = 0; n < n_tiles; ++n) {
      uint8_t* const tile = s_tile + buf * kTileBytes;
      if (++buf == n_bufs) buf = 0;
      bool ok = wait_bar_warp(&sm.abort_flag, &sm.s_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u, fw);
      tcgen05_fence_after();
      float z[8];  // [4 k + 2 c + e]: row 8 k + t_lane + e, column col0 + 8 c
      float nan_sum = 0.f;
      bool need = !ok;
      if (has_cols && ok) {
        uint32_t sr[8];
        tmem_ld_rows8(lane_base + kRows * (n & 1) + 16 * rh, sr);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float s0 = __uint_as_float(sr[4 * (k >> 1) + (k & 1)]), s1 = __uint_as_float(sr[4 * (k >> 1) + 2 + (k & 1)]);
          nan_sum += s0;  // S is bounded: the sum is NaN where a row holds one
          z[4 * (k >> 1) + (k & 1)] = s0 * qs[0];
          z[4 * (k >> 1) + 2 + (k & 1)] = s1 * qs[1];
        }
        if (vis != 15u) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if ((vis >> k & 1u) == 0) z[4 * (k >> 1) + (k & 1)] = z[4 * (k >> 1) + 2 + (k & 1)] = -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
          top[c] = fmaxf(top[c], fmaxf(fmaxf(z[2 * c], z[2 * c + 1]), fmaxf(z[4 + 2 * c], z[4 + 2 * c + 1])));
        // differences, as P's exponent is one: a sum would be rounded to far scores' step
        need = isnan(nan_sum) || top[0] - ref[0] > kRaiseAt || top[1] - ref[1] > kRaiseAt;
      }
      if (!ok) atomicMin(&sm.abort_tile, n);
      // every softmax thread takes the same branch at every barrier: a failed
      // wait is recorded with its tile before that tile's barrier
      if (softmax_any(need)) {
        if (*reinterpret_cast<volatile int*>(&sm.abort_tile) <= n) {
          aborted = true;
          break;
        }
        // A cached row that holds a NaN makes its whole column of S NaN.  Who
        // sees it gets NaN through P; for those that do not, 0 x NaN must not
        // reach O^T, so the row's values leave the tile.
        if (quad == 0 && __any_sync(0xFFFFFFFFu, isnan(nan_sum))) {
          uint32_t sr[8];
          tmem_ld_rows8(lane_base + kRows * (n & 1) + 16 * rh, sr);
          uint32_t rows = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) rows |= isnan(__uint_as_float(sr[4 * (k >> 1) + (k & 1)])) ? 1u << k : 0u;
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            if ((rows >> k & 1u) == 0) continue;
            const int row = 16 * rh + 8 * (k >> 1) + t_lane + (k & 1);
            for (int dg = lane >> 2; dg < kLatent / 8; dg += 8)
              *reinterpret_cast<uint4*>(tile + dg * kDgBytes + row * 16) = make_uint4(0, 0, 0, 0);
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          top[c] = fmaxf(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], 1));
          top[c] = fmaxf(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], 2));
          if ((lane & 3) == 0) sm.part[rh][col0 + 8 * c] = top[c];
        }
        named_bar_sync(3, kSoftmaxThreads);
        if (has_cols) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float m = fmaxf(top[c], sm.part[rh ^ 1][col0 + 8 * c]);
            float al = 1.f;
            if (m - ref[c] > kRaiseTo) {
              float to = m - kRaiseTo;
              to = m - to > kRaiseAt ? m : to;  // at 2^27 the step is 16, which f16 does not hold
              al = ex2(ref[c] - to);            // 0 while nothing has been seen
              ref[c] = to;
            }
            l_part[c] *= al;
            if ((lane & 3) == 0 && rh == 0) sm.alpha[col0 + 8 * c] = al;
          }
        }
        if (n > 0) {
          // O^T's columns lie across all four quadrants: each warp scales its lanes.
          named_bar_sync(3, kSoftmaxThreads);  // alpha is written again behind two more barriers
          const int last = n - 1;  // its O^T must be done; this tile's waits for its P
          ok = wait_bar_warp(&sm.abort_flag, &sm.free_[last % n_bufs], static_cast<uint32_t>(last / n_bufs) & 1u, fw);
          if (!ok) atomicMin(&sm.abort_tile, n + 1);
          tcgen05_fence_after();
          if (ok) {
#pragma unroll 1
            for (int m = rh; m < 4 * (u.ncols / 16); m += 2) {
              const int cg = m >> 2;
              const uint32_t ta = lane_base + kOCol + kCols * (m & 3) + 16 * cg;
              uint32_t o[16];
              tmem_ld16(ta, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * sm.alpha[16 * cg + j]);
              tmem_st16(ta, o);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          }
        }
      }
      if (has_cols) {
        // a masked z is -inf, and so is the reference of a column that has seen nothing
        const float sub[2] = {ref[0] == -INFINITY ? 0.f : ref[0], ref[1] == -INFINITY ? 0.f : ref[1]};
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            // The denominator sums P before its rounding to f16 (operand type of
            // the product): the LSE keeps float accuracy.  Each row's weight in
            // the output is off by at most 2^-11 of itself, or 2^-34 of the
            // largest where that is more.
            const float p0 = ex2(z[4 * k + 2 * c] - sub[c]), p1 = ex2(z[4 * k + 2 * c + 1] - sub[c]);
            l_part[c] += p0 + p1;
            *reinterpret_cast<__half2*>(tile + kPOff + (2 * quad + c) * kPGroupBytes + (2 * rh + k) * 128 +
                                        (lane >> 2) * 16 + 2 * t_lane) = __floats2half2_rn(p0, p1);
          }
      }
      tcgen05_fence_before();
      if (ok) warp_publish(&sm.p_full[n & 1], lane);
      vis = seen_rows(n + 1, id);
      id = tile_id(u, u.begin + n + 2);
    }
    // ---- denominators and LSEs, once every product is done
    const bool ok = !aborted && wait_bar_warp(&sm.abort_flag, &sm.done, 0u, fw);
    if (!ok) atomicMin(&sm.abort_tile, -1);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      l_part[c] += __shfl_xor_sync(0xFFFFFFFFu, l_part[c], 1);
      l_part[c] += __shfl_xor_sync(0xFFFFFFFFu, l_part[c], 2);
      if ((lane & 3) == 0) sm.part[rh][col0 + 8 * c] = l_part[c];
    }
    named_bar_sync(4, kSoftmaxThreads);
    if ((lane & 3) == 0 && has_cols && rh == 0) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = col0 + 8 * c;
        const float l = l_part[c] + sm.part[1][col];
        sm.alpha[col] = l == 0.f ? 0.f : 1.f / l;  // 0 when the column saw nothing
        const float lse2 = l == 0.f ? -INFINITY : ref[c] + lg2(l);
        if (ok && !direct)
          args.part_lse[(u.col0 + col) * args.parts + u.part] = lse2;
        else if (ok && args.lse != nullptr)
          args.lse[u.col0 + col] = lse2 * kLn2f;
      }
    }
  }

  // ---- output: a warp has its quadrant's tensor-memory lanes; the four warps
  // of a quadrant share the pieces of 128 dims x 16 columns
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  if (warp >= kFirstSoftmax && *reinterpret_cast<volatile int*>(&sm.abort_tile) == kNoAbort) {
    const int quad = warp & 3;
#pragma unroll 1
    for (int piece = cw >> 2; piece < 4 * (u.ncols / 16); piece += kWarps / 4) {
      const int m = piece & 3, cg = piece >> 2;
      uint32_t o[16];
      tmem_ld16((static_cast<uint32_t>(32 * quad) << 16) + kOCol + kCols * m + 16 * cg, o);
      const int dim = 128 * m + 32 * quad + lane;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float inv = sm.alpha[16 * cg + j];
        const float x = inv == 0.f ? 0.f : __uint_as_float(o[j]) * inv;
        const int64_t col = u.col0 + 16 * cg + j;
        if (direct)
          args.out[col * kLatent + dim] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
        else
          args.part_o[(col * args.parts + u.part) * kLatent + dim] = x;
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
// Coherent loads from L2: this grid may be resident before the partials are
// written, which the read-only path does not allow.
constexpr int kMergeChunk = 8;
__global__ void __launch_bounds__(128) dense_merge_kernel(const float* __restrict__ part_o,
                                                          const float* __restrict__ part_lse, int parts,
                                                          uint16_t* __restrict__ out, float* __restrict__ lse) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t col = blockIdx.x;
  const int t = threadIdx.x;
  const float* pl = part_lse + col * parts;
  const float4* src = reinterpret_cast<const float4*>(part_o + col * parts * kLatent) + t;
  float mx = -INFINITY, wsum = 0.f;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < parts; s0 += kMergeChunk) {
    float ls[kMergeChunk];
    float4 v[kMergeChunk];
#pragma unroll
    for (int i = 0; i < kMergeChunk; ++i) ls[i] = s0 + i < parts ? __ldcg(pl + s0 + i) : -INFINITY;
#pragma unroll
    for (int i = 0; i < kMergeChunk; ++i)
      v[i] = ls[i] != -INFINITY ? __ldcg(src + static_cast<int64_t>(s0 + i) * (kLatent / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
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
      acc[0] += w * v[i].x;
      acc[1] += w * v[i].y;
      acc[2] += w * v[i].z;
      acc[3] += w * v[i].w;
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
// the prefix's CTAs, with the own rows' CTAs in the SMs that the last of those
// waves leaves idle and in waves of their own after it, + the joining of the
// partials (about four tiles, and one for every 6).  In eighths of a tile; the
// fewest partials among equals.  The own rows' slices are as long as the prefix's,
// or, where that makes more of them than a call without a prefix has, the number
// of that call if it is better: a prefix of one tile must not cut long contexts
// into single tiles (32 requests x 16 heads, 140,000 own rows behind a prefix of
// 500: 274 slices, now 19).
DensePlan plan_dense_decode(int batch, int q_len, int num_heads, int64_t own_rows, int prefix_len) {
  constexpr int64_t kStartTiles = 8;
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
  const int64_t alone = pre_tiles > 0 ? plan_dense_decode(batch, q_len, num_heads, own_rows, 0).splits : 0;
  int64_t best = -1;
  for (int64_t n = 1; n <= tiles && n <= sms; ++n) {
    const int64_t slice = (tiles + n - 1) / n;
    const int64_t waves = (groups * n + sms - 1) / sms;
    auto consider = [&](int64_t s) {  // n slices of the prefix and s of the own rows (0: n of the own rows)
      int64_t cost = 8 * waves * (slice + kStartTiles);
      if (s > 0) {
        const int64_t own_slice = (own_tiles + s - 1) / s;
        const int64_t fit = (waves * sms - groups * n) * ((slice + kStartTiles) / (own_slice + kStartTiles));
        if (own_groups * s > fit) cost += 8 * ((own_groups * s - fit + sms - 1) / sms) * (own_slice + kStartTiles);
      }
      if (n + s > 1) cost += 32 + 4 * (n + s) / 3;
      if (best < 0 || cost < best) {
        best = cost;
        p.prefix_splits = static_cast<int>(s > 0 ? n : 0);
        p.splits = static_cast<int>(s > 0 ? s : n);
      }
    };
    if (pre_tiles == 0) {
      consider(0);
    } else {
      const int64_t match = own_tiles > slice ? (own_tiles + slice - 1) / slice : 1;
      if (match <= sms) consider(match);
      if (match > alone) consider(alone);
    }
    if (groups * n > 4 * sms) break;  // every SM has several CTAs already
  }
  const size_t parts = static_cast<size_t>(p.prefix_splits) + p.splits;
  if (parts > 1)
    p.workspace = (static_cast<size_t>(columns) * parts * ((kLatent + 1) * sizeof(float)) + 255) / 256 * 256;
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
    const size_t o_bytes = static_cast<size_t>(a.columns) * a.parts * kLatent * sizeof(float);
    a.part_o = static_cast<float*>(workspace);
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
  const float* po = a.part_o;
  const float* pl = a.part_lse;
  void* merge[] = {&po, &pl, &a.parts, &a.out, &a.lse};
  return launch_dependent(reinterpret_cast<const void*>(dense_merge_kernel), static_cast<unsigned>(a.columns), 128, 0,
                          merge, stream);
}

}  // namespace mla
