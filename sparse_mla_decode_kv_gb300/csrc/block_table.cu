// Block tables and slot maps from request lengths.
//
// Every request b holds ceil(ctx_b / 64) blocks and gets n_b new tokens:
//   start_b = sum_{a<b} n_a            (exclusive scan over the batch)
//   need_b  = max(0, min(ceil((ctx_b + n_b) / 64), width) - ceil(ctx_b / 64))
//   rank_b  = sum_{a<b} need_a         (exclusive scan)
// its i-th new block is the free ring's entry head + rank_b + i while that is
// before the tail, and token j's slot is its block x 64 + position % 64.
//
// Bound: latency.  The work is two scans over the batch and 12 bytes written
// per token, so every CTA repeats the scans for itself (512 requests at a
// time, one per thread; 8 bytes a request from L2) and then fills its own
// range of tokens and its share of the new table entries: one launch, no
// exchange between CTAs.  A token finds its request by a binary search of the
// starts in shared memory, four independent searches per thread.
#include <cuda_runtime.h>

#include <cstdint>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kTile = 512;     // requests per pass, threads per CTA
constexpr int kPerThread = 4;  // tokens per thread
constexpr int kChunk = kTile * kPerThread;

// Exclusive scan of `x` over the CTA's kTile threads; *total gets the sum.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, off);
    if (lane >= off) inc += y;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kTile / 32; ++w) {
    const int64_t s = warp_sums[w];
    before += w < warp ? s : 0;
    all += s;
  }
  *total = all;
  __syncthreads();  // warp_sums may be written again
  return before + inc - x;
}

// Largest r in [0, kTile) with starts[r] <= x (starts ascending, starts[0] <= x).
__device__ __forceinline__ int find(const int* starts, int x) {
  int r = 0;
#pragma unroll
  for (int step = kTile / 2; step > 0; step >>= 1)
    if (starts[r + step] <= x) r += step;
  return r;
}

// kMap: slots, positions and table entries; kMeta: starts, grown lengths and
// the ring's state (CTA 0).  Both in one launch, unless an output replaces the
// input that other CTAs still read.
template <bool kMap, bool kMeta>
__global__ void __launch_bounds__(kTile) block_table_extend_kernel(const ExtendArgs a) {
  __shared__ int64_t warp_sums[kTile / 32];
  __shared__ int s_start[kTile], s_rank[kTile];  // first token, first new block (within the pass)
  __shared__ int s_ctx[kTile], s_have[kTile];
  __shared__ int64_t s_end[kTile];  // positions below it have a block
  const int tid = threadIdx.x;
  const int64_t head = a.free_state[0], tail = a.free_state[1];
  const int64_t cap = a.free_capacity;
  const int64_t left = head <= tail ? min(tail - head, cap) : 0;  // blocks that can be given
  int64_t at = cap > 0 ? head % cap : 0;
  if (at < 0) at += cap;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kChunk;
  const int64_t c1 = min(c0 + kChunk, a.num_slots);

  // the id of the new block of rank g (counted over the whole batch)
  auto new_block = [&](int64_t g) -> int {
    if (g >= left) return -1;
    int64_t i = at + g;
    if (i >= cap) i -= cap;
    return __ldg(a.free_blocks + i);
  };

  int64_t tokens = 0, blocks = 0;  // before this pass
  for (int r0 = 0; r0 < a.batch; r0 += kTile) {
    const int r = r0 + tid;
    const bool in = r < a.batch;
    const int64_t ctx = in ? max(a.context_lens[r], 0) : 0;
    const int64_t want_new = in ? max(a.new_lens[r], 0) : 0;
    int64_t sum_new, sum_need;
    const int64_t first = min(tokens + block_scan(want_new, warp_sums, &sum_new), a.num_slots);
    const int64_t n = min(want_new, a.num_slots - first);
    const int64_t have = (ctx + kBlock - 1) / kBlock;
    const int64_t want = min((ctx + n + kBlock - 1) / kBlock, static_cast<int64_t>(a.max_blocks));
    const int64_t need = max(want - have, static_cast<int64_t>(0));
    const int64_t rank = block_scan(need, warp_sums, &sum_need);
    const int64_t granted = min(max(left - blocks - rank, static_cast<int64_t>(0)), need);
    const int64_t room = min(have + granted, static_cast<int64_t>(a.max_blocks)) * kBlock;
    const int64_t end = min(min(ctx + n, max(ctx, room)), static_cast<int64_t>(0x7FFFFFFF));
    s_start[tid] = static_cast<int>(first);  // past the batch: the pass's end
    s_rank[tid] = static_cast<int>(rank);
    s_ctx[tid] = static_cast<int>(ctx);
    s_have[tid] = static_cast<int>(have);
    s_end[tid] = end;
    __syncthreads();
    const int64_t pass_end = min(tokens + sum_new, a.num_slots);
    if (kMeta && blockIdx.x == 0 && in) {
      a.query_start[r] = static_cast<int>(first);
      a.context_lens_out[r] = static_cast<int>(end);
    }
    if (kMap) {
      for (int64_t f = static_cast<int64_t>(blockIdx.x) * kTile + tid; f < sum_need;
           f += static_cast<int64_t>(gridDim.x) * kTile) {
        const int q = find(s_rank, static_cast<int>(f));
        a.block_table[static_cast<int64_t>(r0 + q) * a.max_blocks + s_have[q] + (f - s_rank[q])] = new_block(blocks + f);
      }
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) {
        const int64_t t = c0 + i * kTile + tid;
        if (t < tokens || t >= min(pass_end, c1)) continue;
        const int q = find(s_start, static_cast<int>(t));
        const int64_t pos = s_ctx[q] + (t - s_start[q]);
        const int64_t blk = pos / kBlock;
        int id = -1;
        if (pos < s_end[q] && blk < a.max_blocks)
          id = blk < s_have[q] ? a.block_table[static_cast<int64_t>(r0 + q) * a.max_blocks + blk]
                               : new_block(blocks + s_rank[q] + (blk - s_have[q]));
        a.slot_mapping[t] = id >= 0 && id < a.num_blocks ? static_cast<int64_t>(id) * kBlock + pos % kBlock : -1;
        a.positions[t] = pos <= 0x7FFFFFFF ? static_cast<int>(pos) : -1;
      }
    }
    tokens = pass_end;
    blocks += sum_need;
    __syncthreads();  // the pass's tables may be overwritten
  }
  if (kMap) {  // padding behind the last token
    for (int64_t t = max(c0, tokens) + tid; t < c1; t += kTile) {
      a.slot_mapping[t] = -1;
      a.positions[t] = -1;
    }
  }
  if (kMeta && blockIdx.x == 0 && tid == 0) {
    const int64_t taken = min(blocks, left);
    a.query_start[a.batch] = static_cast<int>(tokens);
    a.free_state_out[0] = head + taken;
    a.free_state_out[1] = tail;
    a.free_state_out[2] = blocks - taken;
  }
}

}  // namespace

cudaError_t launch_block_table_extend(const ExtendArgs& a, cudaStream_t stream) {
  const int64_t chunks = (a.num_slots + kChunk - 1) / kChunk;
  const unsigned grid = static_cast<unsigned>(chunks > 0 ? chunks : 1);
  // One CTA reads everything before it writes it back; several would race.
  const bool in_place = a.context_lens_out == a.context_lens || a.free_state_out == a.free_state;
  if (grid == 1 || !in_place) {
    block_table_extend_kernel<true, true><<<grid, kTile, 0, stream>>>(a);
    return cudaGetLastError();
  }
  block_table_extend_kernel<true, false><<<grid, kTile, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  block_table_extend_kernel<false, true><<<1, kTile, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
