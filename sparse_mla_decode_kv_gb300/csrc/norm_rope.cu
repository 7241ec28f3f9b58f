// Norms of queries and keys with the position rotation in the same pass, and
// the same pass writing a latent row into the paged cache.
//
// Per head of D values:  y = x / sqrt(mean(x^2) + eps) * w  (left out without
// a weight), then the 64 values from rope_offset on are rotated in pairs:
//   (x, y) -> (x cos a - y sin a, y cos a + x sin a),   a = position * inv_freq_i
// with pair i the values 2i, 2i + 1 (interleaved) or i, i + 32.
//
// Angles.  position * inv_freq in float loses the angle of far positions
// (2^20 x 2^-24 = 0.06 rad), and FP64 is slow here.  A turn fraction is kept
// instead: inv_freq / 2 pi as a 64-bit fixed-point fraction of a turn, times
// the position modulo 2^64 -- exact integer arithmetic -- whose upper 32 bits
// are the phase to 2^-32 of a turn.  sincospi then sees an argument in [-1, 1].
//
// Latent rows.  The normed latent and the rotated key are rounded to bf16 and
// then quantised exactly as the quantize-on-write kernel quantises bf16 rows:
// the cache holds the bytes that storing this pass's bf16 rows would give, so
// a row does not depend on which way it was written.
//
// Bound: HBM, 4 bytes per query / key value; per latent row 1,152 bytes and 12
// of slot and position in, 352 (NVFP4) or 576 (FP8) out, where a norm pass
// followed by the quantize-on-write pass would move 2,304 bytes more.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kWarps = 8;
constexpr int kPairs = kRope / 2;
constexpr int kHeadsPerTask = 4;  // consecutive (token, head) rows of one lane group, loaded together

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float bf16_rn(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

// sin and cos of position x the pair's frequency (a 64-bit fraction of a turn).
__device__ __forceinline__ void angle(uint64_t turn, int position, float* s, float* c) {
  const uint64_t phase = turn * static_cast<uint64_t>(static_cast<int64_t>(position));
  sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, s, c);  // 2^-31
}

// One lane group (G lanes, 8 values each) per run of heads.
template <int G>
__device__ __forceinline__ void norm_rope_heads(const NormRopeArgs& a, const HeadSet& hs, int64_t task,
                                                const uint64_t* turns) {
  const int lane = threadIdx.x & 31;
  const int gl = lane & (G - 1);
  const int64_t rows = a.tokens * hs.heads;
  const int64_t r0 = task * kHeadsPerTask;
  const bool has = 8 * gl < a.dim;
  const int rc = gl - a.rope_offset / 8;  // 8-value chunk within the rotated part
  const bool turned = rc >= 0 && rc < kRope / 8;
  uint4 x[kHeadsPerTask];
  int64_t tok[kHeadsPerTask];
  int head[kHeadsPerTask];
  tok[0] = rows <= 0x7FFFFFFF ? static_cast<uint32_t>(r0) / static_cast<uint32_t>(hs.heads) : r0 / hs.heads;
  head[0] = static_cast<int>(r0 - tok[0] * hs.heads);
#pragma unroll
  for (int i = 0; i < kHeadsPerTask; ++i) {
    if (i > 0) {
      const bool wrap = head[i - 1] + 1 == hs.heads;
      tok[i] = tok[i - 1] + wrap;
      head[i] = wrap ? 0 : head[i - 1] + 1;
    }
    x[i] = make_uint4(0, 0, 0, 0);
    if (has && r0 + i < rows)
      x[i] = *reinterpret_cast<const uint4*>(hs.in + tok[i] * hs.in_token + head[i] * hs.in_head + 8 * gl);
  }
  uint4 w4 = make_uint4(0, 0, 0, 0);
  if (has && hs.weight != nullptr) w4 = __ldg(reinterpret_cast<const uint4*>(hs.weight) + gl);
  const uint32_t ww[4] = {w4.x, w4.y, w4.z, w4.w};
  int64_t angle_tok = -1;
  // interleaved: this chunk's pairs; else half of them, the other half is the partner's
  float sn[4] = {0.f, 0.f, 0.f, 0.f}, cs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kHeadsPerTask; ++i) {
    const bool in = r0 + i < rows;  // uniform over the lane group
    const uint32_t xw[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = bf16_bits_to_f32(xw[k] & 0xFFFFu);
      v[2 * k + 1] = __uint_as_float(xw[k] & 0xFFFF0000u);
    }
    if (hs.weight != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(v[k], v[k], ss);
#pragma unroll
      for (int off = G / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
      const float rstd = rsqrtf(ss / static_cast<float>(a.dim) + a.eps);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] *= rstd * bf16_bits_to_f32(ww[k] & 0xFFFFu);
        v[2 * k + 1] *= rstd * __uint_as_float(ww[k] & 0xFFFF0000u);
      }
    }
    if (turned && in && tok[i] != angle_tok) {
      angle_tok = tok[i];
      const int pos = __ldg(a.positions + angle_tok);
      const int p0 = a.interleaved ? 4 * rc : 8 * (rc & 3) + (rc & 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) angle(turns[p0 + k], pos, &sn[k], &cs[k]);
    }
    if (a.interleaved) {
      if (turned) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float p = v[2 * k], q = v[2 * k + 1];
          v[2 * k] = p * cs[k] - q * sn[k];
          v[2 * k + 1] = q * cs[k] + p * sn[k];
        }
      }
    } else {
      // chunk rc and its partner rc ^ 4 hold the two halves of 8 pairs and
      // half of their angles each
      const int src = turned ? lane + ((rc & 4) ? -4 : 4) : lane;
      const float sign = (rc & 4) ? 1.f : -1.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float other = __shfl_sync(0xFFFFFFFFu, v[k], src);
        const float so = __shfl_sync(0xFFFFFFFFu, sn[k & 3], src), co = __shfl_sync(0xFFFFFFFFu, cs[k & 3], src);
        const bool mine = (k >> 2) == ((rc >> 2) & 1);
        const float s = mine ? sn[k & 3] : so, c = mine ? cs[k & 3] : co;
        if (turned) v[k] = v[k] * c + sign * other * s;
      }
    }
    if (has && in)
      *reinterpret_cast<uint4*>(hs.out + tok[i] * hs.out_token + head[i] * hs.out_head + 8 * gl) =
          make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
  }
}

// One warp per latent row: lane g owns scale group g (16 latent values) and
// one rotated pair.
template <int FMT>
__device__ __forceinline__ void norm_rope_append_row(const NormRopeArgs& a, int64_t n, const uint64_t* turns) {
  const int lane = threadIdx.x & 31;
  const int64_t slot = __ldg(a.slot_mapping + n);
  const uint16_t* src = a.kv + n * a.kv_token;
  const uint4 v0 = __ldg(reinterpret_cast<const uint4*>(src + lane * kGroup));
  const uint4 v1 = __ldg(reinterpret_cast<const uint4*>(src + lane * kGroup) + 1);
  const int e0 = a.interleaved ? 2 * lane : lane, e1 = a.interleaved ? 2 * lane + 1 : lane + kPairs;
  const float p = bf16_bits_to_f32(__ldg(src + kLatent + e0)), q = bf16_bits_to_f32(__ldg(src + kLatent + e1));
  const int pos = __ldg(a.positions + n);
  const uint4 w0 = __ldg(reinterpret_cast<const uint4*>(a.latent_weight + lane * kGroup));
  const uint4 w1 = __ldg(reinterpret_cast<const uint4*>(a.latent_weight + lane * kGroup) + 1);
  if (slot < 0 || slot / kBlock >= a.num_blocks) return;  // skipped (warp-uniform)
  const uint32_t xw[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  const uint32_t ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  float x[16], ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf16_bits_to_f32(xw[i] & 0xFFFFu);
    x[2 * i + 1] = __uint_as_float(xw[i] & 0xFFFF0000u);
    ss = fmaf(x[2 * i], x[2 * i], ss);
    ss = fmaf(x[2 * i + 1], x[2 * i + 1], ss);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
  const float rstd = rsqrtf(ss * (1.f / kLatent) + a.eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf16_rn(x[2 * i] * (rstd * bf16_bits_to_f32(ww[i] & 0xFFFFu)));
    x[2 * i + 1] = bf16_rn(x[2 * i + 1] * (rstd * __uint_as_float(ww[i] & 0xFFFF0000u)));
  }
  float s, c;
  angle(turns[lane], pos, &s, &c);
  const uint32_t rope2 = f32x2_to_e4m3x2(bf16_rn(q * c + p * s), bf16_rn(p * c - q * s));
  uint8_t* row = a.pool + (slot / kBlock) * a.block_stride + (slot % kBlock) * (FMT == 0 ? kRowNvfp4 : kRowFp8);
  store_latent_row<FMT>(row, lane, x);
  uint8_t* rope = row + (FMT == 0 ? kRopeOffNvfp4 : kRopeOffFp8);
  if (a.interleaved) {
    *reinterpret_cast<uint16_t*>(rope + 2 * lane) = static_cast<uint16_t>(rope2);
  } else {
    rope[lane] = static_cast<uint8_t>(rope2);
    rope[lane + kPairs] = static_cast<uint8_t>(rope2 >> 8);
  }
}

// CTAs [0, kv_ctas) take latent rows, the others tasks of the two head sets.
template <int G>
__global__ void __launch_bounds__(kWarps * 32)
    norm_rope_kernel(const NormRopeArgs a, unsigned kv_ctas, int64_t q_tasks, int64_t tasks) {
  __shared__ uint64_t turns[kPairs];
  if (threadIdx.x < kPairs) {
    // inv_freq / 2 pi of a turn, as a fraction of 2^64
    const double f = a.inv_freq[threadIdx.x] * 0.15915494309189535;
    turns[threadIdx.x] = static_cast<uint64_t>((f - floor(f)) * 18446744073709551616.0);
  }
  __syncthreads();
  if (blockIdx.x < kv_ctas) {
    const int64_t n = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (n >= a.tokens) return;
    if (a.fmt == 0)
      norm_rope_append_row<0>(a, n, turns);
    else
      norm_rope_append_row<1>(a, n, turns);
    return;
  }
  const int64_t task = (static_cast<int64_t>(blockIdx.x - kv_ctas) * (kWarps * 32) + threadIdx.x) / G;
  // whole warps stay together: the shuffles name every lane
  const int64_t warp_first = (static_cast<int64_t>(blockIdx.x - kv_ctas) * (kWarps * 32) + (threadIdx.x & ~31u)) / G;
  if (warp_first >= tasks) return;
  // q_tasks is a multiple of the tasks per warp, so a warp has one set
  const bool is_k = warp_first >= q_tasks;
  norm_rope_heads<G>(a, a.set[is_k], task - (is_k ? q_tasks : 0), turns);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  const int group = a.dim <= 64 ? 8 : a.dim <= 128 ? 16 : 32;  // lanes per head, 8 values each
  const int per_warp = 32 / group;
  int64_t set_tasks[2];
  for (int i = 0; i < 2; ++i) {
    const int64_t rows = a.set[i].in != nullptr ? a.tokens * a.set[i].heads : 0;
    const int64_t t = (rows + kHeadsPerTask - 1) / kHeadsPerTask;
    set_tasks[i] = (t + per_warp - 1) / per_warp * per_warp;
  }
  const int64_t tasks = set_tasks[0] + set_tasks[1];
  const int64_t kv_ctas = a.kv != nullptr ? (a.tokens + kWarps - 1) / kWarps : 0;
  const int64_t head_ctas = (tasks * group + kWarps * 32 - 1) / (kWarps * 32);
  const int64_t grid = kv_ctas + head_ctas;
  if (grid == 0) return cudaSuccess;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  auto* kernel = group == 8 ? norm_rope_kernel<8> : group == 16 ? norm_rope_kernel<16> : norm_rope_kernel<32>;
  kernel<<<static_cast<unsigned>(grid), kWarps * 32, 0, stream>>>(a, static_cast<unsigned>(kv_ctas), set_tasks[0], tasks);
  return cudaGetLastError();
}

}  // namespace mla
