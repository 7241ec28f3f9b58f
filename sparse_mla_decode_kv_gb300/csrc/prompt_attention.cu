// Attention over whole prompts, packed one behind another: causal or full,
// grouped heads, bf16, on the fifth-generation tensor cores.
//
// Mathematics.  Per query head and tile of 128 rows, over tiles of 128 keys:
//   S = Q . K^T,   P = 2^(S scale - r),   O = O + P . V,   l = l + sum P
// with r the row's running maximum, which may lag by 2^8 (P is bf16, whose range
// is float's: a lag costs no precision), and out = O / l, lse = ln 2 (r + log2 l).
// S, O, r and l are float; P is rounded to bf16 as V's partner in the product: a
// key's weight in out is off by at most 2^-8 of itself, in l it is not rounded.
//
// Rows.  The G query heads of a key head share its keys: a tile is 128 / G tokens
// x G heads, so a few tokens of many heads fill it as well as many tokens of one.
//
// Work split.  One CTA has two tiles of one sequence and key head and walks
// (a slice of) their keys; the tensor core works on one tile while the other's
// softmax runs.  Tiles lie in tensor memory: S 2 x 128 columns, O 2 x 128; P
// overlays S as the A operand of its product.  Warp 0 issues the products, warp
// 1 the copies, warps 2 and 3 look through the values that some row must not see,
// and two groups of four warps have a tile's softmax, a thread a row: maximum and
// sum stay in registers.  Products of one issuing thread complete in order, so a
// full S says that the product before it, which read P and V, is done too.
// Slices' partial outputs are joined by their LSEs in a second kernel.
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
constexpr int kMmaWarp = 0, kCopyWarp = 1, kCleanWarp = 2, kFirstSoftmax = 4;
constexpr int kThreads = 12 * 32;
constexpr int kChunkBytes = kTile * 128;  // 128 rows of 64 values
constexpr int kItems = 16;                // barriers of copied tiles (keys and values in turn)
constexpr int kSmemBytes = 227 * 1024;
constexpr int kCtlBytes = 1024;
constexpr uint32_t kSCol = 0, kOCol = 256, kTmemCols = 512;
constexpr float kLag = 8.f;
constexpr float kLn2 = 0.6931471805599453f;
// Tiles of keys that some of a CTA's rows see and others do not: what its up to 256
// tokens see ends within 255 keys of one another, in at most three tiles.
constexpr int kMaskedTiles = 3;
// Registers of the 128 issuing and searching threads, and of the 256 of the softmax:
// together what 384 threads are launched with.
constexpr int kLaunchRegs = 168, kFewRegs = 56, kManyRegs = 224;
static_assert(128 * kFewRegs + 256 * kManyRegs == kThreads * kLaunchRegs, "registers");

struct Ctl {
  uint64_t q_full[2], full[kItems], free_[kItems], s_full[2], p_full[2], o_full[2], done;
  uint64_t masked_full[kMaskedTiles], clean[kMaskedTiles];  // values of masked tiles: copied, searched
  uint32_t tmem_base;
  int abort_flag;
  uint32_t bad[kMaskedTiles][kTile / 32];  // keys of the masked tiles that held an infinity or NaN
  int any_bad;
};
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");

template <int KC>
__host__ __device__ constexpr int ring_chunks() {
  return (kSmemBytes - kCtlBytes - 1024 - 2 * KC * kChunkBytes) / kChunkBytes;
}

__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,"
      "%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,"
      "%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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

// One CTA's part: two tiles of a sequence's query tokens, one key head, tiles of
// keys [begin, begin + count[s]) for tile s.
struct Unit {
  int q0, nq;        // the sequence's first query token and their number
  int k0, nk;
  int tok[2];        // first token of either tile within the sequence
  int head;          // key head
  int begin;
  int count[2];
  int split;
};

template <int KC, int VC>
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

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- which tiles.  Sequence b's pairs of tiles have the places from q_start[b] /
  // tokens + b on: as many as there are places before sequence b + 1's, or fewer.
  const int per = kTile / args.group;  // tokens of a tile
  Unit u;
  u.split = blockIdx.x % args.splits;
  const int rest = blockIdx.x / args.splits;
  u.head = rest % args.kv_heads;
  const int place = args.places - 1 - rest / args.kv_heads;  // the longest rows of a sequence first
  int seq = -1;
  for (int b0 = 0; b0 < args.batch; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    bool before = false;
    if (b < args.batch) {
      const int at = min(max(args.q_start[b], 0), args.q_tokens);
      before = at / (2 * per) + b <= place;
    }
    seq += __syncthreads_count(before);
  }
  if (seq < 0) return;
  u.q0 = min(max(args.q_start[seq], 0), args.q_tokens);
  u.nq = max(0, min(max(args.q_start[seq + 1], 0), args.q_tokens) - u.q0);
  u.k0 = min(max(args.kv_start[seq], 0), args.kv_tokens);
  u.nk = max(0, min(max(args.kv_start[seq + 1], 0), args.kv_tokens) - u.k0);
  u.tok[0] = (place - (u.q0 / (2 * per) + seq)) * 2 * per;
  u.tok[1] = u.tok[0] + per;
  if (u.tok[0] >= u.nq) return;
  // keys that token i of the sequence sees: the first limit(i)
  auto limit = [&](int i) { return args.causal ? min(max(u.nk - u.nq + i + 1, 0), u.nk) : u.nk; };
  {
    int n[2];
    for (int s = 0; s < 2; ++s)
      n[s] = u.tok[s] < u.nq ? (limit(min(u.tok[s] + per, u.nq) - 1) + kTile - 1) / kTile : 0;
    const int64_t all = max(n[0], n[1]);
    u.begin = static_cast<int>(all * u.split / args.splits);
    const int end = static_cast<int>(all * (u.split + 1) / args.splits);
    for (int s = 0; s < 2; ++s) u.count[s] = max(0, min(end, n[s]) - u.begin);
  }
  const int n_tiles = max(u.count[0], u.count[1]);
  // tiles of keys that some row does not see in full, from this one on
  const int first_masked = limit(u.tok[0]) / kTile;
  const int rows = per * args.group;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.o_full[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.free_[i], 1);
    }
    for (int i = 0; i < kMaskedTiles; ++i) {
      mbar_init(&sm.masked_full[i], 1);
      mbar_init(&sm.clean[i], 2);
    }
    mbar_init(&sm.done, 1);
    sm.abort_flag = 0;
    sm.any_bad = 0;
    fence_mbar_init();
  }
  if (threadIdx.x >= 32 && threadIdx.x < 32 + kMaskedTiles * 4)
    sm.bad[(threadIdx.x - 32) >> 2][threadIdx.x & 3] = 0;
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

  // Copied tiles in turn: item 2 j has the keys of tile j, item 2 j + 1 the values.
  // Their chunks follow one another around the ring.
  auto chunk_of = [](int item) { return (item >> 1) * kPairChunks + (item & 1) * KC; };
  // The values of masked tiles, at most the last three of a sequence, have barriers
  // of their own, which the searching warps can wait for from the start.
  auto masked = [&](int j) { return u.begin + j - first_masked; };  // which one tile j is, negative: none
  auto full_bar = [&](int item) {
    return (item & 1) && masked(item >> 1) >= 0 ? &sm.masked_full[masked(item >> 1)] : &sm.full[item % kItems];
  };
  auto full_parity = [&](int item) {
    return (item & 1) && masked(item >> 1) >= 0 ? 0u : static_cast<uint32_t>(item / kItems) & 1u;
  };
  auto item_full = [&](int item) { return wait_bar(sm, full_bar(item), full_parity(item), fw); };

  if (warp < kFirstSoftmax) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == kCopyWarp) {
      // ---------------------------------------------------------- copies
      int issued = 0;  // items whose copy was started
      bool q_issued[2] = {false, false};
      if (elect_one()) {
        auto copy_q = [&](int s) {
          mbar_expect_tx(&sm.q_full[s], static_cast<uint32_t>(KC * rows * 128));
          q_issued[s] = true;
          for (int c = 0; c < KC; ++c)
            tma_load_3d(s_q + (s * KC + c) * kChunkBytes, &q_map, 64 * c, u.head * args.group, u.q0 + u.tok[s],
                        &sm.q_full[s]);
        };
        int freed = 0;  // items known to be free again
        bool ok = true;
        for (int i = 0; i < 2 * n_tiles && ok; ++i) {
          const int chunks = (i & 1) ? VC : KC;
          const int first = chunk_of(i);
          // the items before this one whose places it takes
          while (ok && chunk_of(freed) < first + chunks - kRing) {
            ok = wait_bar(sm, &sm.free_[freed % kItems], static_cast<uint32_t>(freed / kItems) & 1u, fw);
            ++freed;
          }
          if (!ok) break;
          if (i == 0 && u.count[0] > 0) copy_q(0);
          uint64_t* const bar = full_bar(i);
          mbar_expect_tx(bar, static_cast<uint32_t>(chunks * kChunkBytes));
          for (int c = 0; c < chunks; ++c)
            tma_load_3d(s_ring + (first + c) % kRing * kChunkBytes, (i & 1) ? &v_map : &k_map, 64 * c, u.head,
                        u.k0 + (u.begin + (i >> 1)) * kTile, bar);
          issued = i + 1;
          if (i == 0 && u.count[1] > 0) copy_q(1);
        }
        // no copy may be in flight when the CTA leaves
        for (int s = 0; s < 2; ++s)
          if (q_issued[s]) mbar_wait_bounded(&sm.q_full[s], 0u, fw, kFaultPromptWait);
        for (int i = max(0, issued - kItems); i < issued; ++i)
          mbar_wait_bounded(full_bar(i), full_parity(i), fw, kFaultPromptWait);
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------- products
      const uint32_t idesc_s = bf16_idesc(kTile, args.negate, false);
      constexpr uint32_t idesc_o = bf16_idesc(64 * VC, false, true);
      if (elect_one()) {
        const uint64_t q_desc = umma_desc_sw128(smem_u32(s_q));
        const uint32_t ring = smem_u32(s_ring);
        auto scores = [&](int s, int j) {  // S of tile s and keys j
          const int first = chunk_of(2 * j);
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const uint64_t k_desc = umma_desc_sw128(ring + (first + c) % kRing * kChunkBytes);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              umma_ss(kSCol + kTile * s, q_desc + (((s * KC + c) * kChunkBytes + 32 * i) >> 4), k_desc + (32 * i >> 4),
                      idesc_s, c > 0 || i > 0);
          }
          umma_commit(&sm.s_full[s]);
        };
        bool ok = true;
        if (n_tiles > 0) {
          ok = item_full(0);
          for (int s = 0; s < 2 && ok; ++s) {
            if (u.count[s] == 0) continue;
            ok = wait_bar(sm, &sm.q_full[s], 0u, fw);
            if (!ok) break;
            tcgen05_fence_after();
            scores(s, 0);
          }
          umma_commit(&sm.free_[0]);
        }
#pragma unroll 1
        for (int j = 0; j < n_tiles && ok; ++j) {
          ok = item_full(2 * j + 1);
          if (ok && masked(j) >= 0) ok = wait_bar(sm, &sm.clean[masked(j)], 0u, fw);
          if (ok && j + 1 < n_tiles) ok = item_full(2 * j + 2);
          const int v0 = chunk_of(2 * j + 1);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (ok && j < u.count[s]) {
              ok = wait_bar(sm, &sm.p_full[s], static_cast<uint32_t>(j) & 1u, fw);
              if (!ok) break;
              tcgen05_fence_after();
              // the two chunks of a value tile may lie at the ring's two ends
              uint32_t at[VC];
#pragma unroll
              for (int c = 0; c < VC; ++c) at[c] = ring + (v0 + c) % kRing * kChunkBytes;
              if (VC == 1 || at[VC - 1] == at[0] + kChunkBytes) {
                const uint64_t v_desc = desc_values(at[0]);
#pragma unroll
                for (int i = 0; i < kTile / 16; ++i)
                  umma_ts(kOCol + kTile * s, kSCol + kTile * s + 8 * i, v_desc + (2048 * i >> 4), idesc_o, j > 0 || i > 0);
              } else {
#pragma unroll
                for (int c = 0; c < VC; ++c) {
                  const uint64_t v_desc = desc_values(at[c]);
#pragma unroll
                  for (int i = 0; i < kTile / 16; ++i)
                    umma_ts(kOCol + kTile * s + 64 * c, kSCol + kTile * s + 8 * i, v_desc + (2048 * i >> 4),
                            bf16_idesc(64, false, true), j > 0 || i > 0);
                }
              }
              if (j + 1 == u.count[s]) umma_commit(&sm.o_full[s]);
            }
            if (s == 1) umma_commit(&sm.free_[(2 * j + 1) % kItems]);
            if (ok && j + 1 < u.count[s]) scores(s, j + 1);
          }
          if (j + 1 < n_tiles) umma_commit(&sm.free_[(2 * j + 2) % kItems]);
        }
        umma_commit(&sm.done);
        mbar_wait_bounded(&sm.done, 0u, fw, kFaultPromptWait);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- values that are no numbers
      const int half = warp - kCleanWarp;  // keys 64 half ..
      for (int j = max(0, first_masked - u.begin); j < n_tiles; ++j) {
        const int item = 2 * j + 1;
        if (!wait_bar_warp(sm, full_bar(item), 0u, fw)) break;
#pragma unroll 1
        for (int r = 0; r < 2; ++r) {
          const int key = 64 * half + 32 * r + lane;
          uint32_t top = 0;  // the largest magnitudes, two at a time
#pragma unroll
          for (int c = 0; c < VC; ++c) {
            const uint8_t* row = s_ring + (chunk_of(item) + c) % kRing * kChunkBytes + key * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // in another order in each lane, so that they read different banks
              const uint4 v = *reinterpret_cast<const uint4*>(row + 16 * ((i + lane) & 7));
              top = __vmaxu2(__vmaxu2(top, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu)),
                             __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
            }
          }
          const bool bad = (top & 0x7FFFu) >= 0x7F80u || (top >> 16) >= 0x7F80u;
          const uint32_t which = __ballot_sync(0xFFFFFFFFu, bad);
          if (bad) {
            for (int c = 0; c < VC; ++c) {
              uint16_t* row = reinterpret_cast<uint16_t*>(s_ring + (chunk_of(item) + c) % kRing * kChunkBytes + key * 128);
              for (int i = 0; i < 64; ++i)
                if ((row[i] & 0x7F80u) == 0x7F80u) row[i] = 0;
            }
          }
          if (which != 0 && lane == 0) {
            sm.bad[masked(j)][2 * half + r] = which;
            *reinterpret_cast<volatile int*>(&sm.any_bad) = 1;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.clean[masked(j)]);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
    const int s = (warp - kFirstSoftmax) >> 2;
    const int quad = warp & 3;
    const int row = 32 * quad + lane;
    const int tok = u.tok[s] + row / args.group;
    const int head = u.head * args.group + row % args.group;
    const bool here = row < rows && tok < u.nq;
    const int count = u.count[s];
    const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
    const uint32_t s_addr = lanes + kSCol + kTile * s, o_addr = lanes + kOCol + kTile * s;
    const int lim = here ? limit(tok) : 0;
    const int tile_full = u.tok[s] < u.nq ? limit(u.tok[s]) / kTile : 0;  // tiles that all rows see in full
    const float sl = args.scale_log2;
    const uint64_t sl2 = pack2(sl, sl);
    float ref = -INFINITY;  // of the scaled scores, base 2
    uint64_t l2[2] = {0, 0};
    bool ok = true;
#pragma unroll 1
    for (int j = 0; j < count; ++j) {
      ok = wait_bar_warp(sm, &sm.s_full[s], static_cast<uint32_t>(j) & 1u, fw);
      if (!ok) break;
      tcgen05_fence_after();
      uint32_t z[2][64];
      tmem_ld64(s_addr, z[0]);
      tmem_ld64(s_addr + 64, z[1]);
      if (u.begin + j >= tile_full) {
        const int rel = lim - (u.begin + j) * kTile;
#pragma unroll
        for (int i = 0; i < kTile; ++i)
          if (i >= rel) z[i >> 6][i & 63] = 0xFF800000u;
      }
      float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < 64; i += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            m[k] = max3(m[k], __uint_as_float(z[half][i + k]), __uint_as_float(z[half][i + 4 + k]));
      const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * sl;
      const bool raise = top - ref > kLag;
      if (__any_sync(0xFFFFFFFFu, raise)) {
        float alpha = 1.f;
        if (raise) {
          alpha = ex2(ref - top);  // 0 while nothing has been seen
          ref = top;
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
      const float sub = ref == -INFINITY ? 0.f : -ref;
      const uint64_t sub2 = pack2(sub, sub);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t p[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float x, y;
          unpack2(fma2(pack2(__uint_as_float(z[half][2 * i]), __uint_as_float(z[half][2 * i + 1])), sl2, sub2), x, y);
          x = ex2(x);
          y = ex2(y);
          l2[i & 1] = add2(l2[i & 1], pack2(x, y));
          p[i] = bf16x2_rn(x, y);
        }
        tmem_st32(s_addr + 32 * half, p);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[s]);
    }
    // ---- output
    float l;
    {
      float x0, x1, x2, x3;
      unpack2(l2[0], x0, x1);
      unpack2(l2[1], x2, x3);
      l = (x0 + x1) + (x2 + x3);
    }
    if (ok && count > 0) ok = wait_bar_warp(sm, &sm.o_full[s], 0u, fw);
    if (ok && u.tok[s] < u.nq) {
      tcgen05_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t t = u.q0 + tok;
      const bool direct = args.splits == 1;
      const float lse2 = l == 0.f ? -INFINITY : ref + lg2(l);
      const int64_t part = (t * args.heads + head) * args.splits + u.split;
      if (here) {
        if (!direct)
          args.part_lse[part] = lse2;
        else if (args.lse != nullptr)
          args.lse[t * args.heads + head] = lse2 * kLn2;
      }
      const bool bad = *reinterpret_cast<volatile int*>(&sm.any_bad) != 0;
#pragma unroll 1
      for (int c = 0; c < args.dv; c += 32) {
        uint32_t o[32];
        if (count > 0) {
          tmem_load_32cols(o_addr + c, o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0;
        }
        if (bad) {
#pragma unroll 1
          for (int w = 0; w < kMaskedTiles * 4; ++w) {
            uint32_t keys = sm.bad[w >> 2][w & 3];
            while (keys != 0) {
              const int key = (first_masked + (w >> 2)) * kTile + 32 * (w & 3) + __ffs(keys) - 1;
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
            uint4* dst = reinterpret_cast<uint4*>(args.out + t * args.out_token + head * args.out_head + c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c + 8 * i < args.dv)
                dst[i] = make_uint4(bf16x2_rn(__uint_as_float(o[8 * i]), __uint_as_float(o[8 * i + 1])),
                                    bf16x2_rn(__uint_as_float(o[8 * i + 2]), __uint_as_float(o[8 * i + 3])),
                                    bf16x2_rn(__uint_as_float(o[8 * i + 4]), __uint_as_float(o[8 * i + 5])),
                                    bf16x2_rn(__uint_as_float(o[8 * i + 6]), __uint_as_float(o[8 * i + 7])));
          } else if (l != 0.f) {
            uint4* dst = reinterpret_cast<uint4*>(args.part_o + part * args.dv + c);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c + 4 * i < args.dv) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
      }
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

// Joins a (token, head)'s partials, a warp each, four values a lane: LSE = log2
// sum 2^lse_s, out = sum 2^(lse_s - LSE) O_s, in one order.  A partial whose LSE
// is -inf was not written and is not read.  Coherent loads: this grid may be
// resident before the partials are written.
constexpr int kMergeWarps = 4;
__global__ void __launch_bounds__(32 * kMergeWarps) prompt_merge_kernel(const PromptArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t t = at / a.heads;
  const int head = static_cast<int>(at - t * a.heads);
  // tokens before the first sequence and behind the last are left as they are
  if (t < max(__ldcg(a.q_start), 0) || t >= min(__ldcg(a.q_start + a.batch), a.q_tokens)) return;
  float mx = -INFINITY;
  for (int s = 0; s < a.splits; ++s) {
    const float x = __ldcg(a.part_lse + at * a.splits + s);
    mx = x > mx || isnan(x) ? x : mx;
  }
  float sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (mx != -INFINITY) {
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
      const float x = __ldcg(a.part_lse + at * a.splits + s);
      if (x == -INFINITY) continue;
      const float w = ex2(x - mx);
      sum += w;
      if (4 * lane < a.dv) {
        const float4 o = __ldcg(reinterpret_cast<const float4*>(a.part_o + (at * a.splits + s) * a.dv) + lane);
        acc[0] += w * o.x;
        acc[1] += w * o.y;
        acc[2] += w * o.z;
        acc[3] += w * o.w;
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (4 * lane < a.dv)
    *reinterpret_cast<uint2*>(a.out + t * a.out_token + head * a.out_head + 4 * lane) =
        make_uint2(bf16x2_rn(acc[0] * inv, acc[1] * inv), bf16x2_rn(acc[2] * inv, acc[3] * inv));
  if (a.lse != nullptr && lane == 0) a.lse[at] = sum == 0.f ? -INFINITY : (mx + lg2(sum)) * kLn2;
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
                   cudaStream_t stream) {
  const void* kernel = reinterpret_cast<const void*>(prompt_attention_kernel<KC, VC>);
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = set_smem_limit_once(kernel, kSmemBytes, &configured);
  if (e != cudaSuccess) return e;
  void* params[] = {&a, const_cast<CUtensorMap*>(&q), const_cast<CUtensorMap*>(&k), const_cast<CUtensorMap*>(&v)};
  return launch_dependent(kernel, grid, kThreads, kSmemBytes, params, stream);
}

}  // namespace

// How the keys are split: modelled time = full waves of CTAs, each its tiles of
// keys and a start worth four, and the joining of the partials.  Lengths are known
// on the device only: every sequence is taken for an equal share of the tokens.
PromptPlan plan_prompt_attention(int64_t q_tokens, int64_t kv_tokens, int batch, int heads, int kv_heads, int dv) {
  PromptPlan p{};
  const int group = heads / kv_heads;
  const int64_t per = kTile / group;
  p.places = q_tokens / (2 * per) + batch;
  const int64_t used = ((q_tokens + batch - 1) / batch + 2 * per - 1) / (2 * per) * batch;  // places of equal shares
  const int64_t units = (used < p.places ? used : p.places) * kv_heads;
  const int64_t sms = device_sm_count();
  const int64_t tiles = (kv_tokens / batch + kTile - 1) / kTile;
  int64_t best = -1;
  p.splits = 1;
  for (int64_t n = 1; n <= (tiles > 1 ? tiles : 1) && n <= sms; ++n) {
    const int64_t waves = (units * n + sms - 1) / sms;
    const int64_t cost = 8 * waves * ((tiles + n - 1) / n + 4) + (n > 1 ? 24 + 4 * n : 0);
    if (best < 0 || cost < best) {
      best = cost;
      p.splits = static_cast<int>(n);
    }
    if (units * n > 4 * sms) break;
  }
  if (p.splits > 1)
    p.workspace = (static_cast<size_t>(q_tokens) * heads * p.splits * (dv + 1) * sizeof(float) + 255) / 256 * 256;
  return p;
}

cudaError_t launch_prompt_attention(PromptArgs a, const PromptPlan& plan, void* workspace, cudaStream_t stream,
                                    bool* described) {
  a.group = a.heads / a.kv_heads;
  a.splits = plan.splits;
  a.places = static_cast<int>(plan.places);
  a.fault_word = fault_word_ptr();
  *described = true;
  if (a.fault_word == nullptr) return cudaErrorInvalidDevicePointer;
  if (a.splits > 1) {
    a.part_o = static_cast<float*>(workspace);
    a.part_lse = a.part_o + static_cast<size_t>(a.q_tokens) * a.heads * a.splits * a.dv;
  }
  const uint32_t per = static_cast<uint32_t>(kTile / a.group);
  CUtensorMap q, k, v;
  // a tensor without rows is described by one that is never read
  const uint64_t kv_rows = a.kv_tokens > 0 ? static_cast<uint64_t>(a.kv_tokens) : 1;
  const bool have = a.kv_tokens > 0;
  *described = encode_tensor_map_3d(&q, a.q, a.dk, a.heads, a.q_tokens, 2 * a.q_head, 2 * a.q_token, a.group, per) &&
               encode_tensor_map_3d(&k, have ? a.k : a.q, a.dk, a.kv_heads, kv_rows, 2 * a.k_head, 2 * a.k_token, 1, kTile) &&
               encode_tensor_map_3d(&v, have ? a.v : a.q, a.dv, a.kv_heads, kv_rows, 2 * a.v_head, 2 * a.v_token, 1, kTile);
  if (!*described) return cudaSuccess;
  const unsigned grid = static_cast<unsigned>(plan.places * a.kv_heads * a.splits);
  cudaError_t e;
  if (a.dk <= 64 && a.dv <= 64)
    e = launch<1, 1>(a, q, k, v, grid, stream);
  else if (a.dk <= 128)
    e = launch<2, 2>(a, q, k, v, grid, stream);
  else
    e = launch<3, 2>(a, q, k, v, grid, stream);
  if (e != cudaSuccess || a.splits == 1) return e;
  const int64_t pairs = static_cast<int64_t>(a.q_tokens) * a.heads;
  void* merge[] = {&a};
  return launch_dependent(reinterpret_cast<const void*>(prompt_merge_kernel),
                          static_cast<unsigned>((pairs + kMergeWarps - 1) / kMergeWarps), 32 * kMergeWarps, 0, merge,
                          stream);
}

}  // namespace mla
