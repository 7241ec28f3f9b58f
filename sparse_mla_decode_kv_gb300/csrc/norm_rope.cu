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
// the position modulo 2^64 in exact integer arithmetic, of which the upper 32 bits
// are used.  The fraction comes from a double product, so for inv_freq up to 1 the
// phase is within 2^-31 + |position| x 2^-55 of a turn (2^-24 at the ends of 32
// bits).  sincospi then sees an argument in [-1/4, 1/4].
//
// Latent rows.  The normed latent and the rotated key are rounded to bf16 and
// then quantised exactly as the quantize-on-write kernel quantises bf16 rows:
// the cache holds the bytes that storing this pass's bf16 rows would give, so
// a row does not depend on which way it was written.
//
// Bound: HBM, 4 bytes per query / key value; per latent row 1,152 bytes and 12
// of slot and position in, 352 (NVFP4) or 576 (FP8) out, where a norm pass
// followed by the quantize-on-write pass would move 2,304 bytes more.  384,000
// FP8 rows: 123 us, 5,430 GB/s; a second row ahead gains nothing there (124.6),
// nor do more CTAs (48 registers, with spills: 173 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRing = 4;  // rows of a lane group in shared memory: one in work, three on their way
constexpr int kPairs = kRope / 2;
constexpr int kCtasPerSm = 3;  // resident per SM: at 4 the registers spill

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// 4-byte copy, and this thread's copies as groups of which all but the last N have come.
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float bf16_rn(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

// sin and cos of position x the pair's frequency (a 64-bit fraction of a turn).
// The nearest quarter turn is split off as an integer, so that the float holds
// an eighth of a turn at most (half a step of it is 2^-28 of a turn, not 2^-26).
__device__ __forceinline__ void angle(uint64_t turn, int position, float* s, float* c) {
  const uint64_t phase = turn * static_cast<uint64_t>(static_cast<int64_t>(position));
  const uint32_t hi = static_cast<uint32_t>(phase >> 32);
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  float sn, cs;
  sincospif(static_cast<float>(static_cast<int32_t>(hi - (quarter << 30))) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31
  const float x = (quarter & 1) ? cs : sn, y = (quarter & 1) ? sn : cs;
  *s = (quarter & 2) ? -x : x;
  *c = ((quarter + 1) & 2) ? -y : y;
}

// Two floats at a time (the packed forms issue once for both).
struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("{ .reg .b64 p, q; mov.b64 p, {%2, %3}; mov.b64 q, {%4, %5}; mul.rn.f32x2 p, p, q; mov.b64 {%0, %1}, p; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("{ .reg .b64 p, q, r; mov.b64 p, {%2, %3}; mov.b64 q, {%4, %5}; mov.b64 r, {%6, %7}; "
      "fma.rn.f32x2 p, p, q, r; mov.b64 {%0, %1}, p; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ F2 bf16x2_floats(uint32_t two) {
  return {__uint_as_float(two << 16), __uint_as_float(two & 0xFFFF0000u)};
}

// A read-only load that stays where it stands.
__device__ __forceinline__ uint4 load_again(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Eight lanes per head: lane l of them has the 8-value chunks l, l + 8, ... (C
// at most), 128 contiguous bytes a load.  The rotated part is 8 consecutive
// chunks, so every lane has exactly one of them, chunk (l - offset / 8) % 8 of
// the part, and half-split pairs lie in lanes l and l ^ 4.  A lane group takes
// `per` consecutive (token, head) rows and computes the angles of a token once
// for those of its heads that are among them; 4 heads share each instruction.
// Each thread copies its own chunks of the next three rows into shared memory
// while it works on one: 3 CTAs of 256 threads then have 110 KB of reads in
// flight on an SM.  With one row ahead in registers it was 37 KB, and the pass
// over 6,000 tokens x 32 heads x 192 took 33.1 us, then 29.0 (three rows in all
// 33.5, five 29.9, six 34.4; 2 or 4 CTAs 29.2 and 36.7), and 28.2 (147 MB: 5,230
// GB/s) with the first rows on their way before the angles are set up.
template <int C, typename F>
__device__ __forceinline__ void norm_rope_heads(const NormRopeArgs& a, const HeadSet& hs, int64_t task,
                                                int per, const uint64_t* turns, const F& set_turns) {
  extern __shared__ uint4 s_rows[];  // [kRing][C][threads]: each thread's own chunks, then [kRing][threads] positions
  int* const s_pos = reinterpret_cast<int*>(s_rows + kRing * C * kThreads);
  const int gl = threadIdx.x & 7;
  const int64_t rows = a.tokens * hs.heads;
  const int64_t r0 = task * per;
  const int left = static_cast<int>(min(max(rows - r0, static_cast<int64_t>(0)), static_cast<int64_t>(per)));
  const int chunks = a.dim / 8;
  const int off = a.rope_offset / 8;
  const int rc = (gl - off) & 7;              // this lane's chunk within the rotated part
  const int c_rope = (off + rc - gl) / 8;     // and among its own
  const int64_t tok0 = rows <= 0x7FFFFFFF ? static_cast<uint32_t>(r0) / static_cast<uint32_t>(hs.heads) : r0 / hs.heads;
  int head = static_cast<int>(r0 - tok0 * hs.heads), in_head = head;
  const uint16_t* in = hs.in + tok0 * hs.in_token + head * hs.in_head + 8 * gl;
  uint16_t* out = hs.out + tok0 * hs.out_token + head * hs.out_head + 8 * gl;
  const int32_t* pos = a.positions + tok0;
  // row i on its way into the ring, and its token's position with the first of
  // the token's rows
  auto issue = [&](int i) {
    if (i < left) {
      const int slot = i % kRing;
#pragma unroll
      for (int c = 0; c < C; ++c)
        cp_async16(s_rows + (slot * C + c) * kThreads + threadIdx.x, in + (gl + 8 * c < chunks ? 64 * c : 0),
                   gl + 8 * c < chunks ? 16 : 0);
      if (i == 0 || in_head == 0) cp_async4(s_pos + slot * kThreads + threadIdx.x, pos);
      const bool wrap = ++in_head == hs.heads;
      in += wrap ? hs.in_token - (hs.heads - 1) * hs.in_head : hs.in_head;
      pos += wrap;
      in_head = wrap ? 0 : in_head;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) issue(i);
  set_turns();
  const float inv_dim = 1.f / static_cast<float>(a.dim);
  float sn[4], cs[4];  // interleaved: this chunk's pairs; else half of them, the other half is the partner's
#pragma unroll 1
  for (int i = 0; i < per; ++i) {
    const bool here = i < left;  // uniform over the lane group
    const int slot = i % kRing;
    cp_async_wait<kRing - 2>();  // row i has come
    F2 v[C][4];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint4 x = s_rows[(slot * C + c) * kThreads + threadIdx.x];
      v[c][0] = bf16x2_floats(x.x);
      v[c][1] = bf16x2_floats(x.y);
      v[c][2] = bf16x2_floats(x.z);
      v[c][3] = bf16x2_floats(x.w);
    }
    const bool first = i == 0 || head == 0;  // the angles are another token's
    const int at = s_pos[slot * kThreads + threadIdx.x];
    uint16_t* const dst = out;
    const bool wrap = ++head == hs.heads;
    out += wrap ? hs.out_token - (hs.heads - 1) * hs.out_head : hs.out_head;
    head = wrap ? 0 : head;
    issue(i + kRing - 1);
    if (hs.weight != nullptr) {
      F2 ss = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) ss = fma2(v[c][k], v[c][k], ss);
      float s = ss.x + ss.y;
#pragma unroll
      for (int m = 4; m > 0; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
      const float rstd = rsqrtf(s * inv_dim + a.eps);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        // read again for every row (from L1): held, they cost the registers of
        // a third of the warps
        uint4 w = make_uint4(0, 0, 0, 0);
        if (gl + 8 * c < chunks) w = load_again(reinterpret_cast<const uint4*>(hs.weight) + gl + 8 * c);
        v[c][0] = mul2(mul2(v[c][0], F2{rstd, rstd}), bf16x2_floats(w.x));
        v[c][1] = mul2(mul2(v[c][1], F2{rstd, rstd}), bf16x2_floats(w.y));
        v[c][2] = mul2(mul2(v[c][2], F2{rstd, rstd}), bf16x2_floats(w.z));
        v[c][3] = mul2(mul2(v[c][3], F2{rstd, rstd}), bf16x2_floats(w.w));
      }
    }
    if (first && here) {
      const int p0 = a.interleaved ? 4 * rc : 8 * (rc & 3) + (rc & 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) angle(turns[p0 + k], at, &sn[k], &cs[k]);
    }
    F2 r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      r[k] = v[0][k];
#pragma unroll
      for (int c = 1; c < C; ++c) r[k] = c_rope == c ? v[c][k] : r[k];
    }
    if (a.interleaved) {
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = {r[k].x * cs[k] - r[k].y * sn[k], r[k].y * cs[k] + r[k].x * sn[k]};
    } else {
      // chunk rc and its partner rc ^ 4 hold the two halves of 8 pairs and half
      // of their angles each
      const bool upper = (rc & 4) != 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float ox = __shfl_xor_sync(0xFFFFFFFFu, r[k].x, 4), oy = __shfl_xor_sync(0xFFFFFFFFu, r[k].y, 4);
        const int e = 2 * (k & 1);  // values 2 k, 2 k + 1: pairs of the lower or the upper four
        const float s0 = __shfl_xor_sync(0xFFFFFFFFu, sn[e], 4), s1 = __shfl_xor_sync(0xFFFFFFFFu, sn[e + 1], 4);
        const float c0 = __shfl_xor_sync(0xFFFFFFFFu, cs[e], 4), c1 = __shfl_xor_sync(0xFFFFFFFFu, cs[e + 1], 4);
        const bool mine = (k >= 2) == upper;
        const float sx = mine ? sn[e] : s0, sy = mine ? sn[e + 1] : s1;
        const float cx = mine ? cs[e] : c0, cy = mine ? cs[e + 1] : c1;
        r[k] = {r[k].x * cx + (upper ? ox : -ox) * sx, r[k].y * cy + (upper ? oy : -oy) * sy};
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[c][k] = c_rope == c ? r[k] : v[c][k];
      if (here && gl + 8 * c < chunks)
        *reinterpret_cast<uint4*>(dst + 64 * c) =
            make_uint4(bf16x2_rn(v[c][0].x, v[c][0].y), bf16x2_rn(v[c][1].x, v[c][1].y),
                       bf16x2_rn(v[c][2].x, v[c][2].y), bf16x2_rn(v[c][3].x, v[c][3].y));
    }
  }
}

// One warp per latent row: lane g owns scale group g (16 latent values) and
// one rotated pair.  A warp strides over rows and has two in flight: the next
// row's loads are issued before this one's arithmetic.  Weights and the pair's
// frequency stay in registers.
struct LatentRow {
  int64_t slot;
  uint4 v0, v1;
  uint32_t p, q;
  int pos;
};
template <int FMT, typename F>
__device__ __forceinline__ void norm_rope_append_rows(const NormRopeArgs& a, int64_t first, int64_t stride,
                                                      const uint64_t* turns, const F& set_turns) {
  const int lane = threadIdx.x & 31;
  const uint4 w0 = __ldg(reinterpret_cast<const uint4*>(a.latent_weight + lane * kGroup));
  const uint4 w1 = __ldg(reinterpret_cast<const uint4*>(a.latent_weight + lane * kGroup) + 1);
  const uint32_t ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  const int e0 = a.interleaved ? 2 * lane : lane, e1 = a.interleaved ? 2 * lane + 1 : lane + kPairs;
  auto load = [&](int64_t n) {
    LatentRow r;
    r.slot = -1;
    if (n < a.tokens) {
      r.slot = __ldg(a.slot_mapping + n);
      const uint16_t* src = a.kv + n * a.kv_token;
      r.v0 = __ldg(reinterpret_cast<const uint4*>(src + lane * kGroup));
      r.v1 = __ldg(reinterpret_cast<const uint4*>(src + lane * kGroup) + 1);
      r.p = __ldg(src + kLatent + e0);
      r.q = __ldg(src + kLatent + e1);
      r.pos = __ldg(a.positions + n);
    }
    return r;
  };
  LatentRow next = load(first);
  set_turns();
  const uint64_t turn = turns[lane];
  for (int64_t n = first; n < a.tokens; n += stride) {
    const LatentRow r = next;
    next = load(n + stride);
    if (r.slot < 0 || r.slot / kBlock >= a.num_blocks) continue;  // skipped (warp-uniform)
    const uint32_t xw[8] = {r.v0.x, r.v0.y, r.v0.z, r.v0.w, r.v1.x, r.v1.y, r.v1.z, r.v1.w};
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
      const uint32_t two = bf16x2_rn(x[2 * i] * (rstd * bf16_bits_to_f32(ww[i] & 0xFFFFu)),
                                     x[2 * i + 1] * (rstd * __uint_as_float(ww[i] & 0xFFFF0000u)));
      x[2 * i] = bf16_bits_to_f32(two & 0xFFFFu);
      x[2 * i + 1] = __uint_as_float(two & 0xFFFF0000u);
    }
    float s, c;
    angle(turn, r.pos, &s, &c);
    const float p = bf16_bits_to_f32(r.p), q = bf16_bits_to_f32(r.q);
    const uint32_t rope2 = f32x2_to_e4m3x2(bf16_rn(q * c + p * s), bf16_rn(p * c - q * s));
    uint8_t* row = a.pool + (r.slot / kBlock) * a.block_stride + (r.slot % kBlock) * (FMT == 0 ? kRowNvfp4 : kRowFp8);
    store_latent_row<FMT>(row, lane, x);
    uint8_t* rope = row + (FMT == 0 ? kRopeOffNvfp4 : kRopeOffFp8);
    if (a.interleaved) {
      *reinterpret_cast<uint16_t*>(rope + 2 * lane) = static_cast<uint16_t>(rope2);
    } else {
      rope[lane] = static_cast<uint8_t>(rope2);
      rope[lane + kPairs] = static_cast<uint8_t>(rope2 >> 8);
    }
  }
}

// CTAs [0, kv_ctas) take latent rows, the others tasks of the two head sets.
template <int C, int FMT>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm)
    norm_rope_kernel(const NormRopeArgs a, unsigned kv_ctas, int per, int64_t q_tasks, int64_t tasks) {
  __shared__ uint64_t turns[kPairs];
  // Every thread calls this once, after it has started its first loads.
  const auto set_turns = [&] {
    if (threadIdx.x < kPairs) {
      // inv_freq / 2 pi of a turn, as a fraction of 2^64
      const double f = a.inv_freq[threadIdx.x] * 0.15915494309189535;
      turns[threadIdx.x] = static_cast<uint64_t>((f - floor(f)) * 18446744073709551616.0);
    }
    __syncthreads();
  };
  if (FMT >= 0 && blockIdx.x < kv_ctas) {
    norm_rope_append_rows<FMT>(a, static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5),
                               static_cast<int64_t>(kv_ctas) * kWarps, turns, set_turns);
    return;
  }
  if constexpr (C > 0) {
    const int64_t cta = static_cast<int64_t>(blockIdx.x - kv_ctas);
    const int64_t task = (cta * (kWarps * 32) + threadIdx.x) / 8;
    // whole warps stay together: the shuffles name every lane
    const int64_t warp_first = (cta * (kWarps * 32) + (threadIdx.x & ~31u)) / 8;
    if (warp_first >= tasks) {
      set_turns();
      return;
    }
    // q_tasks is a multiple of the tasks per warp, so a warp has one set
    const bool is_k = warp_first >= q_tasks;
    norm_rope_heads<C>(a, a.set[is_k], task - (is_k ? q_tasks : 0), per, turns, set_turns);
  }
}

template <int C>
cudaError_t launch_chunks(const NormRopeArgs& a, unsigned grid, unsigned kv_ctas, int per, int64_t q_tasks, int64_t tasks,
                         cudaStream_t stream) {
  static std::atomic<uint64_t> configured[3];
  const int which = a.kv == nullptr ? 0 : a.fmt == 0 ? 1 : 2;
  auto* kernel = which == 0 ? norm_rope_kernel<C, -1> : which == 1 ? norm_rope_kernel<C, 0> : norm_rope_kernel<C, 1>;
  constexpr int kSmem = C == 0 ? 0 : kRing * kThreads * (C * 16 + 4);
  if (kSmem > 0) {
    const cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(kernel), kSmem, &configured[which]);
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, kThreads, kSmem, stream>>>(a, kv_ctas, per, q_tasks, tasks);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  const int64_t sms = device_sm_count();
  int64_t rows[2], set_tasks[2];
  for (int i = 0; i < 2; ++i) rows[i] = a.set[i].in != nullptr ? a.tokens * a.set[i].heads : 0;
  const int64_t head_rows = rows[0] + rows[1];
  // latent rows: warps that stride over them; beside heads, in a share of the
  // resident CTAs that is their share of the bytes
  const int64_t kv_want = a.kv != nullptr ? (a.tokens + kWarps - 1) / kWarps : 0;
  int64_t kv_cap = sms * kCtasPerSm;
  if (head_rows > 0) {
    const double kv_bytes = static_cast<double>(a.tokens) * ((kLatent + kRope) * 2 + (a.fmt == 0 ? kRowNvfp4 : kRowFp8));
    const double head_bytes = static_cast<double>(head_rows) * a.dim * 4;
    kv_cap = static_cast<int64_t>(sms * kCtasPerSm * (kv_bytes / (kv_bytes + head_bytes))) + 1;
  }
  const int64_t kv_ctas = kv_want < kv_cap ? kv_want : kv_cap;
  // Rows per lane group: all groups resident at once, so that no wave is partly
  // filled, and one row each while they are few (64 tokens x 33 heads: 3.6 us;
  // with 4 rows each 5.6 where this was 4.2).
  const int64_t room = sms * kCtasPerSm - kv_ctas;
  const int64_t groups = (room > 1 ? room : 1) * (kWarps * 4);
  const int64_t per = head_rows > groups ? (head_rows + groups - 1) / groups : 1;
  for (int i = 0; i < 2; ++i) set_tasks[i] = ((rows[i] + per - 1) / per + 3) / 4 * 4;  // whole warps
  const int64_t tasks = set_tasks[0] + set_tasks[1];
  const int64_t head_ctas = (tasks * 8 + kWarps * 32 - 1) / (kWarps * 32);
  const int64_t grid = kv_ctas + head_ctas;
  if (grid == 0) return cudaSuccess;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  if (per > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const unsigned g = static_cast<unsigned>(grid), k = static_cast<unsigned>(kv_ctas);
  const int p = static_cast<int>(per);
  switch (tasks == 0 ? 0 : (a.dim + 63) / 64) {  // 8-value chunks per lane
    case 0: return launch_chunks<0>(a, g, k, p, set_tasks[0], tasks, stream);
    case 1: return launch_chunks<1>(a, g, k, p, set_tasks[0], tasks, stream);
    case 2: return launch_chunks<2>(a, g, k, p, set_tasks[0], tasks, stream);
    case 3: return launch_chunks<3>(a, g, k, p, set_tasks[0], tasks, stream);
    default: return launch_chunks<4>(a, g, k, p, set_tasks[0], tasks, stream);
  }
}

}  // namespace mla
