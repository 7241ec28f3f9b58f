// Attention over whole prompts, packed one behind another: causal or full,
// grouped heads, bf16, on the fifth-generation tensor cores.
//
// Mathematics.  Per query head and tile of 128 rows, over tiles of 128 keys:
//   S = Q . K^T,   P = 2^(S scale - r),   O = O + P . V,   l = l + sum P
// with r 8 above the row's maximum when it was set, and raised when a score passes it: a
// weight is 1 at most, so O leaves float's range no earlier than a sum of weighted
// values does (P is bf16, whose range is float's: the 2^8 cost no precision), and out =
// O / l, lse = ln 2 (r + log2 l).
// S, O, r and l are float; P is rounded to bf16 as V's partner in the product: a
// key's weight in out is off by at most 2^-8 of itself, in l it is not rounded.
//
// Rows.  The G query heads of a key head share its keys: a tile is 128 / G tokens
// x G heads, so a few tokens of many heads fill it as well as many tokens of one.
//
// Work split.  A unit is two tiles of one sequence and key head, or one where two would
// leave SMs idle, and (a slice of) their keys; the tensor core works on one tile while
// the other's softmax runs.
// Tiles lie in tensor memory: S 2 x 128 columns, O 2 x 128; P overlays S as the A
// operand of its product.  A CTA an SM takes units until none is left: the grid
// has one CTA a unit, and a running one cancels the next that has not started and
// takes its place, so the next unit's copies and first products overlap the end of
// this one's.  A warp for each tile issues its products, one finds the units and
// copies, one looks through the values that some row must not see, and two groups
// of four warps have a tile's softmax, a thread a row: maximum and sum stay in
// registers.  A tile's products have one issuing thread and complete in order, so a
// full S says that the product before it, which read P and V, is done too.  Where
// a unit has rows for one tile only, the second tile is the same rows again with
// every other tile of keys, joined in the CTA at the end.  Slices' partial outputs are
// joined by their references and sums in a second kernel.
//
// What bounds it.  Over many keys power (1,380 of 1,400 W) and the chain score,
// softmax, product of each tile, which the other tile's hides in part: 16,384 tokens
// x 16 heads x 192 / 128 causal 805 to 860 us by the GPU, 1,600 to 1,710 TFLOP/s, of 128 /
// 128 693 to 730 us, 1,510 to 1,590; 6,000 x 192 / 128 133 us, 1,380 (the tensor pipe
// active in 61 % of the cycles).
// The same with one CTA a unit 163, units taken in turn 156, a product warp a tile
// and maxima from the loads 144, exponentials in turn 134.  Short prompts (16 packed
// ones of up to 1,500 tokens, 160 us) pay each unit's last softmax and output, 3 to 4
// us; single tokens walk memory: 32 over up to 8,192 keys x 64 / 8 heads 115 us, 5,430
// GB/s (124 with their tiles of keys one after the other); one over 8,192 x 32 / 8 17.
//
// Values that a row must not see.  A weight of 0 does not keep an infinity or
// NaN out of a product.  Where some row's mask cuts a tile of keys, its values are
// searched for them before the product; those found are set to 0 in shared
// memory and added at the end to the rows that do see them.
//
// Every wait is bounded; one that runs out sets the library's fault bit and
// the CTA leaves after its copies and products in flight have drained.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kTile = 128;    // rows of a tile, and keys of one
// Warps 0 and 3 issue the products of tile 0 and 1, warp 1 finds the units and copies,
// warp 2 searches the values.
constexpr int kMmaWarp = 0, kCopyWarp = 1, kCleanWarp = 2, kFirstSoftmax = 4;
constexpr int kThreads = 12 * 32;
constexpr int kChunkBytes = kTile * 128;  // 128 rows of 64 values
constexpr int kItems = 16;                // barriers of copied tiles (keys and values in turn)
constexpr int kUnits = 2;                 // units that are known: one in work, one ahead
constexpr int kSmemBytes = 227 * 1024;
constexpr int kCtlBytes = 2048;
constexpr uint32_t kSCol = 0, kOCol = 256, kTmemCols = 512;
constexpr int kTurnPolls = 40;  // of about 30 cycles
constexpr int64_t kMaxSlice = 65536;  // tiles of keys
constexpr float kLag = 8.f, kLagWeight = 256.f;  // 2^8
// Scaled scores (base 2) from this magnitude on: the rounding that one FMA leaves of a row's largest
// would be an exponent of up to 2^6 and more, and from 2^33 on its weight 0 or infinity.  A row
// with such a score above is NaN, and one that has only such below; beside others those
// have the weight 0 that they should.  (Exact differences for these rows cost the others 5 to
// 25 %: whatever else happens to the scores in registers changes the order of the exponentials.)
constexpr float kFar = 1073741824.f;  // 2^30
constexpr float kLowest = -3.402823466e38f;  // a slice of a row that has only scores below -kFar
constexpr float kLn2 = 0.6931471805599453f;
// Tiles of keys that some of a CTA's rows see and others do not: what its up to 256
// tokens see ends within 255 keys of one another, in at most three tiles.
constexpr int kMaskedTiles = 3;
// Registers of the 128 issuing and searching threads, and of the 256 of the softmax:
// together what 384 threads are launched with.
constexpr int kLaunchRegs = 168, kFewRegs = 104, kManyRegs = 200;
static_assert(128 * kFewRegs + 256 * kManyRegs == kThreads * kLaunchRegs, "registers");

// One or two tiles of a sequence's query tokens, one key head, tiles of keys [begin, begin
// + count[s]) for tile s.
struct Unit {
  int q0, nq;  // the sequence's first query token and their number
  int k0, nk;
  int tok;     // first token of tile 0 within the sequence; tile 1's follow
  int head;    // key head
  int split;
  int begin;
  int count[2];
  int steps;   // tiles of keys that are copied
  int paired;  // tile 1 has tile 0's rows, and every other one of its tiles of keys
  int first_masked;  // tiles of keys from this one on are not seen in full by some row
  int last;          // nothing comes any more
};
struct Ctl {
  uint64_t unit_full[kUnits], unit_free[kUnits];
  uint64_t q_full[2], q_free[2];
  uint64_t full[kItems], free_[kItems];  // copied tiles
  uint64_t ready[kItems / 2];            // values that have been searched
  uint64_t s_full[2], p_full[2][2], o_full[2], done[2], canceled;
  uint4 answer;  // to the request for another unit
  Unit unit[kUnits];
  uint32_t tmem_base;
  int abort_flag;
  uint32_t bad[kUnits][kMaskedTiles][kTile / 32];  // keys of the masked tiles that held an infinity or NaN
  int any_bad[kUnits];
  int busy[2][4];  // a softmax warp is at its exponentials
  uint64_t half_full, half_free;  // the second half of a paired tile: in tensor memory and here, read
  float half_ref[kTile], half_sum[kTile];
};
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");

template <int KC>
__host__ __device__ constexpr int ring_chunks() {
  return (kSmemBytes - kCtlBytes - 1024 - 2 * KC * kChunkBytes) / kChunkBytes;
}

// 64 columns of this warp's 32 lanes and their largest value (NaN left out); complete
// behind tmem_wait.
__device__ __forceinline__ void tmem_ld64_max(uint32_t taddr, uint32_t (&r)[64], float& top) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x64.max.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,"
      "%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,"
      "%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, %64, [%65];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]), "=f"(top)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// All loads of this thread have come; r's first use stays behind it.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[64], float& top) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
        "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
        "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]),
        "+r"(r[32]), "+r"(r[33]), "+r"(r[34]), "+r"(r[35]), "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]),
        "+r"(r[40]), "+r"(r[41]), "+r"(r[42]), "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]),
        "+r"(r[48]), "+r"(r[49]), "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]),
        "+r"(r[56]), "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]), "+r"(r[63]), "+f"(top)
      :
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,"
      "%27,%28,%29,%30,%31,%32};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// One operand from tensor memory, the other from shared memory.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
// bf16 operands, f32 accumulator, M = 128.
__host__ __device__ constexpr uint32_t bf16_idesc(int n, bool negate_a, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (negate_a ? 1u << 13 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kTile >> 4) << 24);
}
// Values: 64 of them are contiguous, 128-byte rows of keys behind one another with
// the 128-byte swizzle, the next 64 a chunk further.
__device__ __forceinline__ uint64_t desc_values(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(kChunkBytes >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
  return e != 0;
}
// Two floats at a time (the packed forms issue once for both).
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ bool wait_slow(int* abort_flag, uint64_t* bar, uint32_t parity, unsigned int* fw) {
  if (mbar_wait_or_abort(bar, parity, abort_flag, fw, kFaultPromptWait)) return true;
  *reinterpret_cast<volatile int*>(abort_flag) = 1;
  return false;
}
__device__ __forceinline__ bool wait_bar(Ctl& sm, uint64_t* bar, uint32_t parity, unsigned int* fw) {
  return mbar_try_wait(bar, parity) || mbar_try_wait(bar, parity) || wait_slow(&sm.abort_flag, bar, parity, fw);
}
__device__ __forceinline__ bool wait_bar_warp(Ctl& sm, uint64_t* bar, uint32_t parity, unsigned int* fw) {
  bool ok = true;
  if (!mbar_try_wait(bar, parity)) ok = wait_bar(sm, bar, parity, fw);
  return __all_sync(0xFFFFFFFFu, ok);
}

// Asks for the next CTA that has not started, to be canceled; the answer comes to
// shared memory.
__device__ __forceinline__ void request_unit(void* answer, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(answer)),
      "r"(smem_u32(bar))
      : "memory");
}
// Its number, or -1: there is none.
__device__ __forceinline__ int requested_unit(const void* answer) {
  int id;
  asm volatile(
      "{ .reg .b128 r; .reg .pred p; .reg .b32 x, y, z, w;\n\t"
      "ld.shared.b128 r, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "mov.b32 x, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {x, y, z, w}, r;\n\t"
      "mov.b32 %0, x; }"
      : "=r"(id)
      : "r"(smem_u32(answer))
      : "memory");
  return id;
}

// Keys that token i of the unit's sequence sees: the first so many.
__device__ __forceinline__ int visible(const PromptArgs& a, int nq, int nk, int i) {
  return a.causal ? min(max(nk - nq + i + 1, 0), nk) : nk;
}
// Unit `id`, found by a whole warp; false if it is empty.  Sequence b's pairs of tiles
// have the places from q_start[b] / tokens + b on: as many as there are places before
// sequence b + 1's, or fewer.
__device__ __forceinline__ bool find_unit(const PromptArgs& a, int id, int lane, bool pairs, Unit& u) {
  const int per = kTile / a.group;  // tokens of a tile
  const int span = pairs ? a.unit_tiles * per : 2 * per;  // and of a unit
  u.split = id % a.splits;
  const int rest = id / a.splits;
  u.head = rest % a.kv_heads;
  const int place = a.places - 1 - rest / a.kv_heads;  // the longest rows of a sequence first
  auto first_place = [&](int b) { return min(max(a.q_start[b], 0), a.q_tokens) / span + b; };
  int lo = -1, hi = a.batch;  // the last b in [lo, hi) whose first place is not behind this one
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int b = lo + (lane + 1) * step;
    const uint32_t before = __ballot_sync(0xFFFFFFFFu, b < hi && first_place(b) <= place);
    lo += __popc(before) * step;
    hi = min(hi, lo + step);
  }
  if (lo < 0) return false;
  u.q0 = min(max(a.q_start[lo], 0), a.q_tokens);
  u.nq = max(0, min(max(a.q_start[lo + 1], 0), a.q_tokens) - u.q0);
  u.k0 = min(max(a.kv_start[lo], 0), a.kv_tokens);
  u.nk = max(0, min(max(a.kv_start[lo + 1], 0), a.kv_tokens) - u.k0);
  u.tok = (place - (u.q0 / span + lo)) * span;
  u.last = 0;
  if (u.tok < 0 || u.tok >= u.nq) return false;
  int n[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int t = u.tok + s * per;
    n[s] = t < u.nq && s * per < span ? (visible(a, u.nq, u.nk, min(t + per, u.nq) - 1) + kTile - 1) / kTile : 0;
  }
  const int64_t all = max(n[0], n[1]);
  u.begin = static_cast<int>(all * u.split / a.splits);
  const int end = static_cast<int>(all * (u.split + 1) / a.splits);
#pragma unroll
  for (int s = 0; s < 2; ++s) u.count[s] = max(0, min(end, n[s]) - u.begin);
  u.steps = max(u.count[0], u.count[1]);
  u.paired = pairs && (span == per || (u.tok + per >= u.nq && u.steps > 1));
  if (u.paired) {
    u.count[0] = (u.steps + 1) / 2;
    u.count[1] = u.steps / 2;
  }
  u.first_masked = visible(a, u.nq, u.nk, u.tok) / kTile;
  return true;
}

// Turns: the two tiles' exponentials take turns, see there.  Pairs: where a sequence's rows
// fill one tile at most, the other one has the same rows and every second tile of keys.
template <int KC, int VC, PromptVariant kVariant>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attention_kernel(const PromptArgs args, const __grid_constant__ CUtensorMap q_map,
                            const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ uint8_t smem_any[];
  uint8_t* const smem_raw = smem_any + ((1024u - (smem_u32(smem_any) & 1023u)) & 1023u);
  Ctl& sm = *reinterpret_cast<Ctl*>(smem_raw);
  uint8_t* const s_q = smem_raw + kCtlBytes;  // [tile][64 dims][128 rows x 128 bytes], swizzled
  uint8_t* const s_ring = s_q + 2 * KC * kChunkBytes;
  constexpr int kRing = ring_chunks<KC>();
  constexpr int kPairChunks = KC + VC;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned int* fw = args.fault_word;

  if (threadIdx.x == 32 * kCopyWarp)
    for (const CUtensorMap* m : {&q_map, &k_map, &v_map})
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  const int per = kTile / args.group, rows = per * args.group;  // tokens and rows of a tile
  if (threadIdx.x == 0) {
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&sm.unit_full[i], 1);
      mbar_init(&sm.unit_free[i], 3 + 8);  // both products' warps, the searching one, the softmax's
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_free[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i][0], 4);
      mbar_init(&sm.p_full[i][1], 4);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.done[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.free_[i], 2);
    }
    for (int i = 0; i < kItems / 2; ++i) mbar_init(&sm.ready[i], 1);
    mbar_init(&sm.canceled, 1);
    mbar_init(&sm.half_full, 4);
    mbar_init(&sm.half_free, 4);
    sm.abort_flag = 0;
    for (int i = 0; i < 8; ++i) sm.busy[i >> 2][i & 3] = 0;
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
  asm volatile("griddepcontrol.wait;" ::: "memory");  // inputs may be written until here
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Copied tiles in turn, over all units: an even item has the keys of a tile, the next
  // one its values.  Their chunks follow one another around the ring.
  auto parity = [](int item) { return static_cast<uint32_t>(item / kItems) & 1u; };
  auto unit_parity = [](int i) { return static_cast<uint32_t>(i / kUnits) & 1u; };

  if (warp < kFirstSoftmax) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == kCopyWarp) {
      // ---------------------------------------------------------- units and copies
      const bool leader = elect_one();
      int issued = 0, freed = 0;  // items (the leader's)
      int at = 0, at_freed = 0;   // first chunk of the next item, and of the next that will be free
      uint32_t q_uses[2] = {0, 0};
      int id = blockIdx.x, n = 0;
      bool ok = true;
      for (uint32_t asked = 0; ok && id >= 0; ++asked) {
        Unit u;
        if (find_unit(args, id, lane, kVariant == kPromptPairs, u)) {
          if (n >= kUnits) ok = wait_bar_warp(sm, &sm.unit_free[n % kUnits], unit_parity(n - kUnits), fw);
          if (ok && leader) {
            sm.unit[n % kUnits] = u;
            sm.any_bad[n % kUnits] = 0;
            for (int i = 0; i < kMaskedTiles * (kTile / 32); ++i) sm.bad[n % kUnits][0][i] = 0;
            mbar_arrive(&sm.unit_full[n % kUnits]);
            const int items = 2 * (kVariant == kPromptPairs ? u.steps : max(u.count[0], u.count[1]));
            auto copy_q = [&](int s) {
              if (q_uses[s] > 0) ok = wait_bar(sm, &sm.q_free[s], (q_uses[s] - 1) & 1u, fw);
              if (!ok) return;
              mbar_expect_tx(&sm.q_full[s], static_cast<uint32_t>(KC * rows * 128));
              ++q_uses[s];
              for (int c = 0; c < KC; ++c)
                tma_load_3d(s_q + (s * KC + c) * kChunkBytes, &q_map, 64 * c, u.head * args.group,
                            u.q0 + u.tok + (kVariant == kPromptPairs && u.paired ? 0 : s * per), &sm.q_full[s]);
            };
            for (int i = 0; i < items && ok; ++i) {
              const int chunks = (i & 1) ? VC : KC;
              // the items before this one whose places it takes
              while (ok && at_freed < at + chunks - kRing) {
                ok = wait_bar(sm, &sm.free_[freed % kItems], parity(freed), fw);
                at_freed += (freed & 1) ? VC : KC;
                ++freed;
              }
              if (!ok) break;
              uint64_t* const bar = &sm.full[issued % kItems];
              mbar_expect_tx(bar, static_cast<uint32_t>(chunks * kChunkBytes));
              for (int c = 0; c < chunks; ++c)
                tma_load_3d(s_ring + (at + c) % kRing * kChunkBytes, (i & 1) ? &v_map : &k_map, 64 * c, u.head,
                            u.k0 + (u.begin + (i >> 1)) * kTile, bar);
              ++issued;
              at += chunks;
              if (at >= 2 * kRing && at_freed >= kRing) {  // both count from the same round of the ring
                at -= kRing;
                at_freed -= kRing;
              }
              if (i == 0) {
                if (u.count[0] > 0) copy_q(0);
                if (ok && u.count[1] > 0) copy_q(1);
              }
            }
          }
          __syncwarp();
          ok = __all_sync(0xFFFFFFFFu, ok);
          ++n;
        }
        if (!ok) break;
        // The next unit is asked for when this one's last copies have been started, two
        // or three tiles before its end: a long unit's successor is for whoever is free
        // first (asked for at once, 6000 tokens x 16 heads took 172 us for 156).
        if (leader) {
          mbar_expect_tx(&sm.canceled, 16);
          request_unit(&sm.answer, &sm.canceled);
        }
        __syncwarp();
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&sm.canceled, asked & 1u, fw, kFaultPromptWait));
        id = requested_unit(&sm.answer);
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (ok && n >= kUnits) ok = wait_bar_warp(sm, &sm.unit_free[n % kUnits], unit_parity(n - kUnits), fw);
      if (leader) {
        if (ok) {
          sm.unit[n % kUnits].last = 1;
          mbar_arrive(&sm.unit_full[n % kUnits]);
        }
        // no copy may be in flight when the CTA leaves
        for (int s = 0; s < 2; ++s)
          if (q_uses[s] > 0) mbar_wait_bounded(&sm.q_full[s], (q_uses[s] - 1) & 1u, fw, kFaultPromptWait);
        for (int i = max(0, issued - kItems); i < issued; ++i)
          mbar_wait_bounded(&sm.full[i % kItems], parity(i), fw, kFaultPromptWait);
      }
      __syncwarp();
    } else if (warp != kCleanWarp) {
      // ---------------------------------------------------------- products of tile s
      const int s = warp == kMmaWarp ? 0 : 1;
      const uint32_t idesc_s = bf16_idesc(kTile, args.negate, false);
      constexpr uint32_t idesc_o = bf16_idesc(64 * VC, false, true);
      if (elect_one()) {
        const uint64_t q_desc = umma_desc_sw128(smem_u32(s_q) + s * KC * kChunkBytes);
        const uint32_t ring = smem_u32(s_ring);
        const uint32_t d_s = kSCol + kTile * s, d_o = kOCol + kTile * s;
        int item = 0, at = 0;  // the unit's first item and its first chunk's place in the ring
        uint32_t q_uses = 0, p_uses = 0;
        bool ok = true;
#pragma unroll 1
        for (int n = 0; ok; ++n) {
          ok = wait_bar(sm, &sm.unit_full[n % kUnits], unit_parity(n), fw);
          if (!ok || sm.unit[n % kUnits].last) break;
          const int count = s == 0 ? sm.unit[n % kUnits].count[0] : sm.unit[n % kUnits].count[1];
          const int n_tiles = kVariant == kPromptPairs ? sm.unit[n % kUnits].steps
                                              : max(count, s == 0 ? sm.unit[n % kUnits].count[1] : sm.unit[n % kUnits].count[0]);
          // of a paired unit's tiles of keys every other one is this tile's
          const bool paired = kVariant == kPromptPairs && sm.unit[n % kUnits].paired;
          auto ours = [&](int j) { return paired ? (j & 1) == s : j < count; };
          auto nth = [&](int j) { return paired ? j >> 1 : j; };
          mbar_arrive(&sm.unit_free[n % kUnits]);
          if (n_tiles == 0) continue;
          auto scores = [&](int j, int k_at) {  // S of keys j, which begin at chunk k_at
#pragma unroll
            for (int c = 0; c < KC; ++c) {
              const int chunk = k_at + c >= kRing ? k_at + c - kRing : k_at + c;
              const uint64_t k_desc = umma_desc_sw128(ring + chunk * kChunkBytes);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                umma_ss(d_s, q_desc + ((c * kChunkBytes + 32 * i) >> 4), k_desc + (32 * i >> 4), idesc_s, c > 0 || i > 0);
            }
            umma_commit(&sm.s_full[s]);
            if (nth(j) + 1 == count) umma_commit(&sm.q_free[s]);
          };
          ok = wait_bar(sm, &sm.full[item % kItems], parity(item), fw);
          if (ok && count > 0) {
            ok = wait_bar(sm, &sm.q_full[s], q_uses & 1u, fw);
            ++q_uses;
            if (ok && ours(0)) {
              tcgen05_fence_after();
              scores(0, at);
            }
          }
          umma_commit(&sm.free_[item % kItems]);
#pragma unroll 1
          for (int j = 0; j < n_tiles && ok; ++j) {
            const int v_item = item + 1, k_item = item + 2;
            int v_at = at + KC, k_at = at + kPairChunks;
            v_at = v_at >= kRing ? v_at - kRing : v_at;
            k_at = k_at >= kRing ? k_at - kRing : k_at;
            ok = wait_bar(sm, &sm.ready[v_item / 2 % (kItems / 2)], parity(v_item), fw);
            if (ok && ours(j)) {
              // the product of the first half of the keys runs while the other's weights
              // are computed
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                if (ok) ok = wait_bar(sm, &sm.p_full[s][half], p_uses & 1u, fw);
                if (!ok) continue;
                tcgen05_fence_after();
                // the two chunks of a value tile may lie at the ring's two ends
                const uint32_t v0 = ring + v_at * kChunkBytes;
                if (VC == 1 || v_at + 1 < kRing) {
                  const uint64_t v_desc = desc_values(v0);
#pragma unroll
                  for (int i = 4 * half; i < 4 * half + 4; ++i)
                    umma_ts(d_o, d_s + 8 * i, v_desc + (2048 * i >> 4), idesc_o, nth(j) > 0 || i > 0);
                } else {
#pragma unroll
                  for (int c = 0; c < VC; ++c) {
                    const uint64_t v_desc = desc_values(c == 0 ? v0 : ring);
#pragma unroll
                    for (int i = 4 * half; i < 4 * half + 4; ++i)
                      umma_ts(d_o + 64 * c, d_s + 8 * i, v_desc + (2048 * i >> 4), bf16_idesc(64, false, true),
                              nth(j) > 0 || i > 0);
                  }
                }
              }
              ++p_uses;
              if (ok && nth(j) + 1 == count) umma_commit(&sm.o_full[s]);
            }
            umma_commit(&sm.free_[v_item % kItems]);
            if (ok && j + 1 < n_tiles) {
              ok = wait_bar(sm, &sm.full[k_item % kItems], parity(k_item), fw);
              if (ok && ours(j + 1)) scores(j + 1, k_at);
              umma_commit(&sm.free_[k_item % kItems]);
            }
            item += 2;
            at = k_at;
          }
        }
        umma_commit(&sm.done[s]);
        mbar_wait_bounded(&sm.done[s], 0u, fw, kFaultPromptWait);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- values that are no numbers
      int item = 1, at = KC;  // the next values and the place of their first chunk in the ring
      bool ok = true;
      for (int n = 0; ok; ++n) {
        ok = wait_bar_warp(sm, &sm.unit_full[n % kUnits], unit_parity(n), fw);
        if (!ok || sm.unit[n % kUnits].last) break;
        const Unit& u = sm.unit[n % kUnits];
        const int n_tiles = kVariant == kPromptPairs ? u.steps : max(u.count[0], u.count[1]);
        const int masked0 = u.first_masked - u.begin;  // tiles from this one on
        const int seen = visible(args, u.nq, u.nk, u.tok);  // keys before it are seen by all rows
        for (int j = 0; j < n_tiles && ok; ++j) {
          ok = wait_bar_warp(sm, &sm.full[item % kItems], parity(item), fw);
          if (!ok) break;
          if (j >= masked0) {
#pragma unroll 1
            for (int r = max(0, seen - (u.begin + j) * kTile) / 32; r < kTile / 32; ++r) {
              const int key = 32 * r + lane;
              const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
              __nv_bfloat162 sum[4] = {zero, zero, zero, zero};  // of products with 0: NaN where there is one
#pragma unroll
              for (int c = 0; c < VC; ++c) {
                const uint8_t* row = s_ring + (at + c >= kRing ? at + c - kRing : at + c) * kChunkBytes + key * 128;
#pragma unroll
                for (int i = 0; i < 8; ++i) {  // in another order in each lane, so that they read different banks
                  const uint4 v = *reinterpret_cast<const uint4*>(row + 16 * ((i + lane) & 7));
                  const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
                  for (int k = 0; k < 4; ++k) sum[k] = __hfma2(x[k], zero, sum[k]);
                }
              }
              const __nv_bfloat162 all = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
              const bool bad = __hisnan(all.x) || __hisnan(all.y);
              const uint32_t which = __ballot_sync(0xFFFFFFFFu, bad);
              if (bad) {
                for (int c = 0; c < VC; ++c) {
                  uint16_t* row = reinterpret_cast<uint16_t*>(
                      s_ring + (at + c >= kRing ? at + c - kRing : at + c) * kChunkBytes + key * 128);
                  for (int i = 0; i < 64; ++i)
                    if ((row[i] & 0x7F80u) == 0x7F80u) row[i] = 0;
                }
              }
              if (which != 0 && lane == 0) {
                sm.bad[n % kUnits][j - masked0][r] = which;
                *reinterpret_cast<volatile int*>(&sm.any_bad[n % kUnits]) = 1;
              }
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.ready[item / 2 % (kItems / 2)]);
          item += 2;
          at += kPairChunks;
          at = at >= kRing ? at - kRing : at;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.unit_free[n % kUnits]);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
    const int s = (warp - kFirstSoftmax) >> 2;
    const int quad = warp & 3;
    const int row = 32 * quad + lane;
    const int row_tok = row / args.group, row_head = row - row_tok * args.group;
    const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
    const uint32_t s_addr = lanes + kSCol + kTile * s, o_addr = lanes + kOCol + kTile * s;
    const float sl = args.scale_log2;
    const uint64_t sl2 = pack2(sl, sl);
    uint32_t s_uses = 0, o_uses = 0, pairs = 0;
    bool ok = true;
#pragma unroll 1
    for (int n = 0; ok; ++n) {
      ok = wait_bar_warp(sm, &sm.unit_full[n % kUnits], unit_parity(n), fw);
      if (!ok || sm.unit[n % kUnits].last) break;
      const Unit& u = sm.unit[n % kUnits];
      const int count = s == 0 ? u.count[0] : u.count[1];
      const bool paired = kVariant == kPromptPairs && u.paired;
      const int tok0 = u.tok + (paired ? 0 : s * per), tok = tok0 + row_tok;
      const int head = u.head * args.group + row_head;
      const bool here = row < rows && tok < u.nq;
      const int lim = here ? visible(args, u.nq, u.nk, tok) : 0;
      const int begin = u.begin;
      const int tile_full = tok0 < u.nq ? visible(args, u.nq, u.nk, tok0) / kTile : 0;  // tiles that all rows see in full
      float ref = -INFINITY;  // of the scaled scores, base 2
      uint64_t l2[2] = {0, 0};
#pragma unroll 1
      for (int j = 0; j < count; ++j) {
        ok = wait_bar_warp(sm, &sm.s_full[s], s_uses & 1u, fw);
        ++s_uses;
        if (!ok) break;
        tcgen05_fence_after();
        uint32_t z[2][64];
        float most[2];
        tmem_ld64_max(s_addr, z[0], most[0]);
        tmem_ld64_max(s_addr + 64, z[1], most[1]);
        tmem_wait(z[0], most[0]);
        tmem_wait(z[1], most[1]);
        const int at_key = begin + (paired ? 2 * j + s : j);  // tile of keys
        if (at_key >= tile_full) {
          const int rel = lim - at_key * kTile;
          most[0] = most[1] = -INFINITY;
#pragma unroll
          for (int i = 0; i < kTile; ++i) {
            if (i >= rel) z[i >> 6][i & 63] = 0xFF800000u;
            most[i & 1] = fmaxf(most[i & 1], __uint_as_float(z[i >> 6][i & 63]));
          }
        }
        const float top = fmaxf(most[0], most[1]) * sl;
        const bool raise = top > ref;
        if (__any_sync(0xFFFFFFFFu, raise)) {
          float alpha = 1.f;
          if (raise && top > -kFar) {
            alpha = ex2(ref - (top + kLag));  // 0 while nothing has been seen
            ref = top + kLag;
            if (!(top < kFar)) alpha = NAN;  // stays in the sum
          }
          const uint64_t a2 = pack2(alpha, alpha);
          l2[0] = fma2(l2[0], a2, 0);
          l2[1] = fma2(l2[1], a2, 0);
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < 64 * VC; c += 32) {
              uint32_t o[32];
              tmem_load_32cols(o_addr + c, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(o_addr + c, o);
            }
          }
        }
        // The two tiles' warps of a scheduler take turns, so that one tile's exponentials run
        // beside the other's products and not beside its exponentials.  A hint: who has
        // waited long enough goes on.  It pays over many tiles of keys (x 16 heads, with
        // and without): 16,384 tokens of 192 dims 805 and 868 us, of 128 693 and 767, 6,000
        // of 192 134 and 142; 2 x 4,096 of 128 124 and 118, 2 x 3,000 of 192 91 and 85.
        if (kVariant == kPromptTurns) {
          for (int i = 0; i < kTurnPolls && *reinterpret_cast<volatile int*>(&sm.busy[s ^ 1][quad]) != 0; ++i) {
          }
          if (lane == 0) *reinterpret_cast<volatile int*>(&sm.busy[s][quad]) = 1;
        }
        const float sub = ref == -INFINITY ? 0.f : -ref;
        const uint64_t sub2 = pack2(sub, sub);
        auto publish = [&](int half) {
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tcgen05_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full[s][half]);
        };
#pragma unroll
        for (int part = 0; part < 4; ++part) {
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int at = 32 * (part & 1) + 2 * i;
            float x, y;
            unpack2(fma2(pack2(__uint_as_float(z[part >> 1][at]), __uint_as_float(z[part >> 1][at + 1])), sl2, sub2), x, y);
            x = ex2(x);
            y = ex2(y);
            l2[i & 1] = add2(l2[i & 1], pack2(x, y));
            p[i] = bf16x2_rn(x, y);
          }
          // the first half is given away a quarter later: its stores are over by then
          if (part == 2) publish(0);
          tmem_st16(s_addr + 16 * part, p);
        }
        if (kVariant == kPromptTurns && lane == 0) *reinterpret_cast<volatile int*>(&sm.busy[s][quad]) = 0;
        publish(1);
      }
      // ---- output
      float l;
      {
        float x0, x1, x2, x3;
        unpack2(l2[0], x0, x1);
        unpack2(l2[1], x2, x3);
        l = (x0 + x1) + (x2 + x3);
      }
      if (ok && count > 0) {
        ok = wait_bar_warp(sm, &sm.o_full[s], o_uses & 1u, fw);
        ++o_uses;
      }
      // A paired tile's halves are joined as slices are: the second one's group leaves its
      // maximum and sum, the first one's reads both sums of values.
      float mine = 1.f, others = 0.f;  // weights of the halves
      if (paired) {
        if (s == 1) {
          sm.half_ref[row] = ref;
          sm.half_sum[row] = l;
          tcgen05_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.half_full);
          if (ok) ok = wait_bar_warp(sm, &sm.half_free, pairs & 1u, fw);
        } else if (ok) {
          ok = wait_bar_warp(sm, &sm.half_full, pairs & 1u, fw);
          const float ref2 = sm.half_ref[row], most = fmaxf(ref, ref2);
          mine = ref == -INFINITY ? 0.f : ex2(ref - most);
          others = ref2 == -INFINITY ? 0.f : ex2(ref2 - most);
          l = mine * l + others * sm.half_sum[row];  // a NaN in either (no score was a number) stays
          ref = most;
        }
        ++pairs;
      }
      if (ok && tok0 < u.nq && !(paired && s == 1)) {
        tcgen05_fence_after();
        const bool lost = l == 0.f && lim > begin * kTile;  // keys are seen, and none has a weight
        const float inv = lost ? NAN : l == 0.f ? 0.f : 1.f / l;
        const int64_t t = u.q0 + tok;
        const bool direct = args.splits == 1;
        const int64_t part = (t * args.heads + head) * args.splits + u.split;
        if (here) {
          if (!direct)
            args.part_lse[part] = lost       ? make_float2(kLowest, kLowest)
                                  : l == 0.f ? make_float2(-INFINITY, -INFINITY)
                                             : make_float2(ref, lg2(l * kLagWeight));
          else if (args.lse != nullptr)
            args.lse[t * args.heads + head] = lost ? NAN : l == 0.f ? -INFINITY : (ref - kLag + lg2(l * kLagWeight)) * kLn2;
        }
        const bool bad = *reinterpret_cast<volatile int*>(&sm.any_bad[n % kUnits]) != 0;
#pragma unroll 1
        for (int c = 0; c < args.dv; c += 32) {
          uint32_t o[32];
          if (paired) {
            uint32_t o2[32];
            tmem_load_32cols(o_addr + c, o);
            tmem_load_32cols(o_addr + kTile + c, o2);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float x = mine == 0.f ? 0.f : mine * __uint_as_float(o[i]);
              o[i] = __float_as_uint(others == 0.f ? x : fmaf(others, __uint_as_float(o2[i]), x));
            }
          } else if (count > 0) {
            tmem_load_32cols(o_addr + c, o);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0;
          }
          if (bad) {
#pragma unroll 1
            for (int w = 0; w < kMaskedTiles * 4; ++w) {
              uint32_t keys = sm.bad[n % kUnits][w >> 2][w & 3];
              while (keys != 0) {
                const int key = (u.first_masked + (w >> 2)) * kTile + 32 * (w & 3) + __ffs(keys) - 1;
                keys &= keys - 1;
                if (key >= lim) break;
                const uint16_t* v = args.v + (u.k0 + key) * args.v_token + u.head * args.v_head + c;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  if (c + i >= args.dv) break;
                  const uint32_t x = v[i];
                  if ((x & 0x7F80u) == 0x7F80u) o[i] = __float_as_uint(__uint_as_float(o[i]) + bf16_bits_to_f32(x));
                }
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = inv == 0.f ? 0u : __float_as_uint(__uint_as_float(o[i]) * inv);
          if (here) {
            if (direct) {
              uint16_t* dst = args.out + t * args.out_token + head * args.out_head + c;
              uint32_t h[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) h[i] = bf16x2_rn(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
              if (args.out_wide) {  // a whole sector a store: half the time of 16-byte ones
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (c + 16 * i < args.dv)
                    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 16 * i), "r"(h[8 * i]),
                                 "r"(h[8 * i + 1]), "r"(h[8 * i + 2]), "r"(h[8 * i + 3]), "r"(h[8 * i + 4]),
                                 "r"(h[8 * i + 5]), "r"(h[8 * i + 6]), "r"(h[8 * i + 7])
                                 : "memory");
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (c + 8 * i < args.dv)
                    *reinterpret_cast<uint4*>(dst + 8 * i) = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
              }
            } else if (l != 0.f) {
              float* dst = args.part_o + part * args.dv + c;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (c + 8 * i < args.dv)
                  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 8 * i), "r"(o[8 * i]),
                               "r"(o[8 * i + 1]), "r"(o[8 * i + 2]), "r"(o[8 * i + 3]), "r"(o[8 * i + 4]),
                               "r"(o[8 * i + 5]), "r"(o[8 * i + 6]), "r"(o[8 * i + 7])
                               : "memory");
            }
          }
        }
      }
      // the tensor memory has been read, by this unit's last loads or its next ones' wait
      tcgen05_fence_before();
      __syncwarp();
      if (paired && s == 0 && lane == 0) mbar_arrive(&sm.half_free);
      if (lane == 0) mbar_arrive(&sm.unit_free[n % kUnits]);
    }
  }

  // ---- no copy or product is in flight any more: their issuers have waited
  tcgen05_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tcgen05_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sm.tmem_base), "r"(kTmemCols) : "memory");
  }
}

// Joins a (token, head)'s partials, a warp each, four values a lane: with slice s's
// reference r_s and l_s = log2 of its sum x 2^8, weights 2^(r_s - R + l_s - L) of the largest R
// and L (apart, as their sum in a float would round a slice's weight by 2^-24 of R), out =
// sum of weight O_s / sum of weights, in one order.  A partial whose l_s is -inf was not
// written and has no part in it, nor one of kLowest unless there are no others: the row is
// NaN.  Coherent loads: this grid may be resident before the partials are written.  What
// bounds it is three round trips to L2, made one (a token x 32 heads over 8,192 keys in 16
// slices 23.2 us before, now 17.2).
constexpr int kMergeWarps = 4;
__global__ void __launch_bounds__(32 * kMergeWarps) prompt_merge_kernel(const PromptArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t t = at / a.heads;
  const int head = static_cast<int>(at - t * a.heads);
  // The bounds, the LSEs (a lane a slice) and the first slices' partials are asked for at once;
  // what was not written is dropped.
  constexpr int kFirst = 8;
  const bool in = t < a.q_tokens, mine = 4 * lane < a.dv;
  const int first = __ldcg(a.q_start), last = __ldcg(a.q_start + a.batch);
  const float2* const lse = a.part_lse + at * a.splits;
  const float* const part = a.part_o + at * a.splits * a.dv + 4 * lane;
  const float2 none = make_float2(-INFINITY, -INFINITY);
  const float2 x0 = in && lane < a.splits ? __ldcg(lse + lane) : none;
  float4 o[kFirst];
#pragma unroll
  for (int s = 0; s < kFirst; ++s) {
    o[s] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in && mine && s < a.splits) o[s] = __ldcg(reinterpret_cast<const float4*>(part + s * a.dv));
  }
  // tokens before the first sequence and behind the last are left as they are
  if (t < max(first, 0) || t >= min(last, a.q_tokens)) return;
  float mx = x0.x, ml = x0.y;  // NaN above all
  for (int s = 32 + lane; s < a.splits; s += 32) {
    const float2 x = __ldcg(lse + s);
    mx = fmaxf(mx, x.x);
    ml = x.y > ml || isnan(x.y) ? x.y : ml;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
    const float x = __shfl_xor_sync(0xFFFFFFFFu, ml, d);
    ml = x > ml || isnan(x) ? x : ml;
  }
  float sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  auto add = [&](float w, float4 v) {
    if (w == 0.f) return;  // not written, or nothing of it is left
    sum += w;
    acc[0] += w * v.x;
    acc[1] += w * v.y;
    acc[2] += w * v.z;
    acc[3] += w * v.w;
  };
  if (mx == kLowest) {
    sum = NAN;
  } else if (ml != -INFINITY) {
    auto weight = [&](float2 x) { return x.y == -INFINITY ? 0.f : ex2((x.x - mx) + (x.y - ml)); };
    const float w0 = weight(x0);
#pragma unroll
    for (int s = 0; s < kFirst; ++s) add(s < a.splits ? __shfl_sync(0xFFFFFFFFu, w0, s) : 0.f, o[s]);
    for (int s0 = 0; s0 < a.splits; s0 += 32) {
      const float w = s0 == 0 ? w0 : weight(s0 + lane < a.splits ? __ldcg(lse + s0 + lane) : none);
      const int n = min(32, a.splits - s0);
#pragma unroll 8
      for (int s = s0 == 0 ? kFirst : 0; s < n; ++s) {
        const float ws = __shfl_sync(0xFFFFFFFFu, w, s);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ws != 0.f && mine) v = __ldcg(reinterpret_cast<const float4*>(part + (s0 + s) * a.dv));
        add(ws, v);
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (4 * lane < a.dv)
    *reinterpret_cast<uint2*>(a.out + t * a.out_token + head * a.out_head + 4 * lane) =
        make_uint2(bf16x2_rn(acc[0] * inv, acc[1] * inv), bf16x2_rn(acc[2] * inv, acc[3] * inv));
  if (a.lse != nullptr && lane == 0) a.lse[at] = sum == 0.f ? -INFINITY : (mx - kLag + (ml + lg2(sum))) * kLn2;
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

template <int KC, int VC>
cudaError_t launch(PromptArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, unsigned grid,
                   PromptVariant variant, cudaStream_t stream) {
  const void* kernel = variant == kPromptTurns ? reinterpret_cast<const void*>(prompt_attention_kernel<KC, VC, kPromptTurns>)
                       : variant == kPromptPairs
                           ? reinterpret_cast<const void*>(prompt_attention_kernel<KC, VC, kPromptPairs>)
                           : reinterpret_cast<const void*>(prompt_attention_kernel<KC, VC, kPromptPlain>);
  static std::atomic<uint64_t> configured[3];
  const cudaError_t e = set_smem_limit_once(kernel, kSmemBytes, &configured[variant]);
  if (e != cudaSuccess) return e;
  void* params[] = {&a, const_cast<CUtensorMap*>(&q), const_cast<CUtensorMap*>(&k), const_cast<CUtensorMap*>(&v)};
  return launch_dependent(kernel, grid, kThreads, kSmemBytes, params, stream);
}

}  // namespace

// How many tiles of rows a unit has, and how its keys are split: modelled time in tiles
// of keys.  Up to a unit an SM, a slice (half of one and the halves' joining where both
// tiles have the same rows) and a start worth three; else the SMs' share of all slices
// and starts, and a slice at the end, when others have run out.  The partials' joining is
// a launch worth two tiles and their bytes (a tile takes about 1.7 us, in which memory
// writes and reads 10 MB).  Units of one tile leave fewer SMs idle: 7 x 33 tokens x 28 / 4
// heads over 315 keys 11.3 us (13.2 with two), 3 x 200 x 4 / 2 over 6,000 21.3 (23.9).
// Lengths are known on the device only: every sequence is taken for an equal share of
// the tokens.
PromptPlan plan_prompt_attention(int64_t q_tokens, int64_t kv_tokens, int batch, int heads, int kv_heads, int dv) {
  PromptPlan p{};
  const int group = heads / kv_heads;
  const int64_t per = kTile / group;
  const int64_t sms = device_sm_count();
  const int64_t tiles = (kv_tokens / batch + kTile - 1) / kTile;
  const int64_t share = (q_tokens + batch - 1) / batch;  // tokens of a sequence
  const double rows_mb = static_cast<double>(q_tokens) * heads * (dv + 2) * 8e-6;  // of one slice, written and read
  double best = -1;
  p.splits = 1;
  for (int unit = 2; unit >= 1; --unit) {  // tiles of rows
    const int64_t places = q_tokens / (unit * per) + batch;
    const int64_t used = (share + unit * per - 1) / (unit * per) * batch;  // of equal shares
    const int64_t units = (used < places ? used : places) * kv_heads;
    // unequal shares may need a place more each: a second round would cost as much as the first
    // (2 sequences of up to 300 tokens x 8 heads over up to 2,000 keys: 7 slices 26.2 us, 6 21.6)
    const int64_t most = batch == 1 ? units : places * kv_heads;
    const bool paired = share <= per;
    for (int64_t n = 1; n <= (tiles > 1 ? tiles : 1) && n <= sms; ++n) {
      const int64_t slice = (tiles + n - 1) / n;
      double cost = static_cast<double>(slice) + 3;
      if ((unit == 1 || paired) && slice > 1) cost = static_cast<double>((slice + 1) / 2) + 3.5;
      if (most * n > sms) {
        if (unit == 1) break;  // more units than SMs: the keys are read for two tiles at once
        cost = static_cast<double>(units * (tiles + 3 * n)) / static_cast<double>(sms) + static_cast<double>(slice);
      }
      if (n > 1) cost += 2 + rows_mb * static_cast<double>(n) * 0.1;
      if (best < 0 || cost < best) {
        best = cost;
        p.splits = static_cast<int>(n);
        p.unit_tiles = unit;
        p.places = places;
      }
      if (units * n > 8 * sms) break;
    }
  }
  // A tile without rows waits for as long as the other's whole slice: no slice may last as
  // long as a bounded wait (a tile of keys takes about 2 us, the longest slice so 0.15 s; the
  // wait gave up after 1.1 s where nothing ever came).
  const int64_t least = ((kv_tokens + kTile - 1) / kTile + kMaxSlice - 1) / kMaxSlice;
  if (p.splits < least) p.splits = static_cast<int>(least);
  // turns: both tiles filled, and 40 tiles of keys a slice or more, on average (without and with:
  // 700 tokens x 16 heads of 192 over 5,200 keys in 3 slices 48 and 52 us, 2,600 x 20 of 64 over
  // 5,400 in 2 105 and 112); pairs: at most one tile
  // filled, and more than one tile of keys (32 single tokens over up to 8,192 keys x 64 / 8
  // heads 114.8 us, 123.9 without; where no unit is paired they cost 3 %)
  const int64_t rows = q_tokens * group;
  const int64_t slice_keys = 1LL * kTile * batch * p.splits;  // a tile of keys for every slice
  p.variant = p.unit_tiles == 2 && rows >= 2LL * kTile * batch && kv_tokens >= 40 * slice_keys ? kPromptTurns
              : p.unit_tiles == 1 || (rows <= 1LL * kTile * batch && kv_tokens > slice_keys)   ? kPromptPairs
                                                                                             : kPromptPlain;
  if (p.splits > 1)
    p.workspace = (static_cast<size_t>(q_tokens) * heads * p.splits * (dv + 2) * sizeof(float) + 255) / 256 * 256;
  return p;
}

cudaError_t launch_prompt_attention(PromptArgs a, const PromptPlan& plan, void* workspace, cudaStream_t stream,
                                    bool* described) {
  a.group = a.heads / a.kv_heads;
  a.splits = plan.splits;
  a.unit_tiles = plan.unit_tiles;
  a.places = static_cast<int>(plan.places);
  a.fault_word = fault_word_ptr();
  a.out_wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.dv % 16 == 0 && (a.q_tokens == 1 || a.out_token % 16 == 0) &&
               (a.heads == 1 || a.out_head % 16 == 0);
  *described = true;
  if (a.fault_word == nullptr) return cudaErrorInvalidDevicePointer;
  if (a.splits > 1) {
    a.part_o = static_cast<float*>(workspace);
    a.part_lse = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(a.q_tokens) * a.heads * a.splits * a.dv);
  }
  const uint32_t per = static_cast<uint32_t>(kTile / a.group);
  CUtensorMap q, k, v;
  // a tensor without rows is described by one that is never read
  const uint64_t kv_rows = a.kv_tokens > 0 ? static_cast<uint64_t>(a.kv_tokens) : 1;
  const bool have = a.kv_tokens > 0;
  const uint64_t kv_heads = have ? static_cast<uint64_t>(a.kv_heads) : 1;
  *described = encode_tensor_map_3d(&q, a.q, a.dk, a.heads, a.q_tokens, 2 * a.q_head, 2 * a.q_token, a.group, per) &&
               encode_tensor_map_3d(&k, have ? a.k : a.q, a.dk, kv_heads, kv_rows, 2 * a.k_head, 2 * a.k_token, 1, kTile) &&
               encode_tensor_map_3d(&v, have ? a.v : a.q, a.dv, kv_heads, kv_rows, 2 * a.v_head, 2 * a.v_token, 1, kTile);
  if (!*described) return cudaSuccess;
  const unsigned grid = static_cast<unsigned>(plan.places * a.kv_heads * a.splits);
  cudaError_t e;
  if (a.dk <= 64 && a.dv <= 64)
    e = launch<1, 1>(a, q, k, v, grid, plan.variant, stream);
  else if (a.dk <= 128)
    e = launch<2, 2>(a, q, k, v, grid, plan.variant, stream);
  else
    e = launch<3, 2>(a, q, k, v, grid, plan.variant, stream);
  if (e != cudaSuccess || a.splits == 1) return e;
  const int64_t pairs = static_cast<int64_t>(a.q_tokens) * a.heads;
  void* merge[] = {&a};
  return launch_dependent(reinterpret_cast<const void*>(prompt_merge_kernel),
                          static_cast<unsigned>((pairs + kMergeWarps - 1) / kMergeWarps), 32 * kMergeWarps, 0, merge,
                          stream);
}

}  // namespace mla
