// Products of a few tokens with matrices of 4-bit weights:
//   y[t, g, n] = W_g * sum_k x[t, g, k] * code[g, n, k] * scale[g, n, k / 16]
// with e2m1 codes and one e4m3 scale per 16 of them (the cache's own latent
// format), x in bf16 or in e4m3 with a float scale per 128 values or per row.
//
// Mathematics.  code * scale has at most 6 significant bits between 2^-10 and
// 2^12: an f16 operand holds it exactly.  e4m3 values are f16 as they are;
// bf16 ones are multiplied by the power of two that brings the largest of their
// 128 to [2^14, 2^15) (a value 2^-29 of it and smaller loses bits past 2^-39 of
// it).  The products of 128 values are added up by the tensor core in float,
// then multiplied by the token's factor for them (its scale, or the power of
// two back) into a float total.
//
// Split.  A CTA has R consecutive rows, as many as make the CTAs equal, and up to 8
// CTAs of a cluster a slice of k each: WR warps share the rows, WK the slice.  A
// warp has 16 rows as the A operand and 8 NT tokens as B
// (m16n8k16), 128 values of k (a piece) a step.  Which 16 values of k an MMA adds
// up is free as long as both operands agree: lane t of a row's four has the 32
// consecutive codes 32 t .. of a piece, so a lane's codes are one 16-byte load, its
// scales one 2-byte load, and every group's scale is needed by one lane only.  The
// tokens lie in shared memory in the order in which the lanes read them.
// Sums of warps and CTAs are joined in one order: a call gives the same bits
// every time.
//
// Bound: HBM, 9/16 byte a weight, and for these matrices latency and the unpacking.
// Memory latency is the first stall (four tokens: long_scoreboard 4.5 warps an issue, 51 %
// of the issue slots used, 35 % of the warps resident).  16 rows x 128 values take a warp
// 107 instructions with up to 8 tokens, 64 cycles of an SM: 4.6 to 4.8 TB/s where memory
// gives 6.8 (without the scales' multiplications 5.8), plus 4 us of start and end.  One
// token x 12288 x 6144 14.4 us, 2,950 GB/s; x 128,000 x 6144 97 us, 4,560; four x 24583 x
// 6144 25.2 us, 3,390.  With 32 tokens it is 290 instructions and 150 cycles (the tokens'
// conversion, the products): x 6144 x 12288 28.7 us.
//
// The weights' way to L2 is not started as a whole while the tokens are laid out.  That
// takes 5 % off 9 to 32 e4m3 tokens (32 x 6144 x 12288 28.1 to 26.6 us, x 12288 x 6144 28.7
// to 27.2), but adds 10 to 13 % to as many bf16 ones, whose layout takes longer (x 6144 x
// 6144 19.4 to 21.3, x 8192 x 16384 44.4 to 49.2), 6 % to four and 18 % to the 128,000 rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kPiece = 128;    // values of k per step of a warp
__host__ __device__ constexpr int stage_tasks(int nt) { return nt == 1 ? 256 : 512; }  // (piece, token) pairs of a stage
constexpr int kMaxRows = 1024;  // of a CTA
constexpr int kMaxSplits = 8;  // portable cluster size
constexpr int kSmemBytes = 227 * 1024;

// By the tiles of 8 tokens: CTAs an SM that registers leave room for, and pieces whose
// weights a warp loads at a time.
__host__ __device__ constexpr int warp_bits(int nt) { return nt == 1 ? 3 : 4; }
__host__ __device__ constexpr int resident(int nt) { return nt == 1 ? 3 : 1; }
__host__ __device__ constexpr int batch(int nt) { return nt == 4 ? 2 : 4; }
// Tokens' values of one piece, in units of 8: [n-tile][4][tokens x 4 lanes] with the
// four 2 units further apart than that, so that a token's sixteen units fall into
// different banks when they are written.  `toks` is a power of two, or 8 NT.
__host__ __device__ constexpr int row_units(int nt, int toks) { return (nt > 1 ? 8 : toks) * 4 + 2; }
__host__ __device__ constexpr int piece_bytes(int nt, int toks) {
  return nt * 4 * row_units(nt, toks) * 16 + (toks < 4 ? 16 : 4 * toks);
}
// e4m3 tokens stay as they are, [token][128 values a piece, and 16 bytes so that two tokens'
// 16-byte reads do not meet], with their factors behind.
constexpr int kRawPad = 16;
__host__ __device__ constexpr int raw_piece_bytes(int toks) { return toks * (kPiece + 4); }
// Joined sums: [WK][tokens][rows, and 4 to spread the banks] floats.
__host__ __device__ constexpr int64_t sum_bytes(int toks, int wk, int64_t rows) { return wk * toks * (rows + 4) * 4; }

struct Weights {  // one lane's part of 16 rows x 128 values: rows g and g + 8
  uint4 code[2];
  uint32_t scale[2];
};

__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t load_two(const uint8_t* p) {
  uint16_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}
// The first product of a sum: nothing to add to.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

template <int NT, bool kCodes>
__global__ void __launch_bounds__(32 << warp_bits(NT), resident(NT)) fp4_matvec_kernel(const MatvecArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kTokens = 8 * NT;
  constexpr int kBatch = batch(NT);
  // A piece's registers are loaded again as soon as it has been used up; with 24 warps an
  // SM (one token tile) that gains nothing.
  constexpr bool kAhead = NT > 1;
  constexpr int kWarpBits = warp_bits(NT), kThreads = 32 << kWarpBits;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int wr_bits = a.row_warps_bits, wk_bits = kWarpBits - wr_bits;
  const int w_row = warp & ((1 << wr_bits) - 1), w_k = warp >> wr_bits, wk = 1 << wk_bits;
  const int block = blockIdx.x / static_cast<unsigned>(a.splits), split = blockIdx.x - block * a.splits;
  const int64_t row0 = static_cast<int64_t>(block) * a.rows;
  const int rows_cta = static_cast<int>(min(static_cast<int64_t>(a.rows), a.n - row0));
  const int grp = blockIdx.y;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.z) * kTokens;
  const int toks = static_cast<int>(min(static_cast<int64_t>(kTokens), a.tokens - tok0));

  // this warp's rows: whole tiles of 16, spread over the warps
  const int tiles = (rows_cta + 15) / 16;
  const int tile0 = (tiles * w_row) >> wr_bits, n_tiles = ((tiles * (w_row + 1)) >> wr_bits) - tile0;
  // the CTA's pieces of k, and of a stage of them this warp's
  const int pieces = (a.k + kPiece - 1) / kPiece;
  const int p_lo = min(split * a.slice, pieces), p_hi = min(p_lo + a.slice, pieces);
  auto stage_lo = [&](int s) { return p_lo + s * a.stage; };
  auto stage_n = [&](int s) { return min(a.stage, p_hi - stage_lo(s)); };
  auto share_lo = [&](int s) { return (stage_n(s) * w_k) >> wk_bits; };
  auto share_n = [&](int s) { return ((stage_n(s) * (w_k + 1)) >> wk_bits) - share_lo(s); };
  const int64_t code_row = a.k / 2, scale_row = a.k / 16;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- tokens.  Half a warp has one token's piece, 8 values a lane.
  const int tok_bits = toks <= 1 ? 0 : 32 - __clz(toks - 1);
  const int tok_p = NT > 1 ? kTokens : 1 << tok_bits;  // tokens with a place
  const int ru = row_units(NT, tok_p);
  uint4* const s_x = reinterpret_cast<uint4*>(smem);
  const int raw_pitch = a.stage * kPiece + kRawPad;
  float* const s_mul = reinterpret_cast<float*>(smem + (kCodes ? tok_p * raw_pitch : a.stage * NT * 4 * ru * 16));  // [piece][token]
  float* const s_sum = reinterpret_cast<float*>(
      smem + (kCodes ? a.stage * raw_piece_bytes(tok_p) + tok_p * kRawPad : a.stage * piece_bytes(NT, tok_p)));  // [w_k][token][row]
  const int pitch = a.rows + 4;
  const int u = lane & 15;
  const uint32_t half = lane & 16 ? 0xFFFF0000u : 0x0000FFFFu;  // the halves may go different ways
  // Tokens that are not there leave what the memory holds: theirs are columns of their
  // own, which nobody reads.
  auto stage_tokens = [&](int s) {
    const int lo = stage_lo(s), n = stage_n(s);
    if constexpr (kCodes) {
      for (int i = threadIdx.x; i < n * toks; i += kThreads) {
        const int tok = i / n, piece = i - tok * n;
        s_mul[piece * tok_p + tok] =
            a.x_scales[((tok0 + tok) * a.groups + grp) * a.x_scale_groups + (a.x_scale_groups > 1 ? lo + piece : 0)];
      }
      const int chunks = n * (kPiece / 16);
      for (int tok = warp; tok < toks; tok += kThreads / 32) {
        const uint8_t* src = static_cast<const uint8_t*>(a.x) + (tok0 + tok) * a.x_token + grp * a.x_group;
        for (int c = lane; c < chunks; c += 32) {
          const int64_t k0 = static_cast<int64_t>(lo) * kPiece + 16 * c;
          const bool in = k0 < a.k;  // zeros behind the end of k
          cp_async16(smem + tok * raw_pitch + 16 * c, in ? src + k0 : src, in ? 16 : 0);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
      const int count = n << tok_bits;
      constexpr int kLoads = 8;
#pragma unroll 1
      for (int i0 = threadIdx.x >> 4; i0 < count; i0 += kLoads * (kThreads / 16)) {
        uint4 raw[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const int i = i0 + j * (kThreads / 16);
          const int tok = i & ((1 << tok_bits) - 1), piece = lo + (i >> tok_bits);
          const int64_t k0 = static_cast<int64_t>(piece) * kPiece + 8 * u;
          raw[j] = make_uint4(0, 0, 0, 0);
          if (i < count && tok < toks && k0 < a.k)
            raw[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + (tok0 + tok) * a.x_token +
                                                     grp * a.x_group + k0);
        }
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const int i = i0 + j * (kThreads / 16);
          const int tok = i & ((1 << tok_bits) - 1), slot = i >> tok_bits;
          if (i >= count) continue;
          uint32_t mx = bf16x8_absmax_bits(raw[j]);
#pragma unroll
          for (int m = 8; m > 0; m >>= 1) mx = max(mx, __shfl_xor_sync(half, mx, m));
          const int shift = query_shift(mx);
          const float up = pow2f(shift);
          const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 p = __floats2half2_rn(bf16_bits_to_f32(w[e] & 0xFFFFu) * up, bf16_bits_to_f32(w[e] >> 16) * up);
            h[e] = *reinterpret_cast<const uint32_t*>(&p);
          }
          s_x[((slot * NT + (tok >> 3)) * 4 + (u & 3)) * ru + (tok & 7) * 4 + (u >> 2)] = make_uint4(h[0], h[1], h[2], h[3]);
          if (u == 0) s_mul[slot * tok_p + tok] = pow2f(-shift);
        }
      }
    }
  };
  for (int i = threadIdx.x; i < wk * tok_p * pitch; i += kThreads) s_sum[i] = 0.f;
  const bool x_here = NT > 1 || g < tok_p;      // else this lane's token (of B) has no place
  const bool y_here = NT > 1 || 2 * t < tok_p;  // and its two tokens of the sums

  const int x_step = kCodes ? kPiece : NT * 4 * ru * 16;  // bytes of a piece's tokens
  float tot[NT][4];
  // One piece: its weights and the tokens of place x (of factors m) into the sums.
  auto add_piece = [&](const Weights& w, const uint8_t* x, const float* m) {
    float acc[NT][4];
    uint32_t sc[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sc[h][0] = e4m3x2_to_f16x2(__byte_perm(w.scale[h], 0, 0x4400));
      sc[h][1] = e4m3x2_to_f16x2(__byte_perm(w.scale[h], 0, 0x4411));
    }
    uint4 raw[kCodes ? NT : 1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 b[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (kCodes) {
          if (j % 2 == 0) raw[n] = *reinterpret_cast<const uint4*>(x + 8 * n * raw_pitch + 8 * j);
          uint32_t lo2[2], hi2[2];
          e4m3x4_to_f16x2x2(j % 2 == 0 ? raw[n].x : raw[n].z, lo2);
          e4m3x4_to_f16x2x2(j % 2 == 0 ? raw[n].y : raw[n].w, hi2);
          b[n] = make_uint4(lo2[0], lo2[1], hi2[0], hi2[1]);
        } else {
          b[n] = *reinterpret_cast<const uint4*>(x + (n * 4 + j) * ru * 16);
        }
        // a token without a place has read another's
        if (NT == 1 && !x_here) b[n] = make_uint4(0, 0, 0, 0);
      }
      const uint4 c0 = w.code[0], c1 = w.code[1];
      uint32_t lo[4], hi[4];
      e2m1x8_to_f16x2x4(j == 0 ? c0.x : j == 1 ? c0.y : j == 2 ? c0.z : c0.w, lo);
      e2m1x8_to_f16x2x4(j == 0 ? c1.x : j == 1 ? c1.y : j == 2 ? c1.z : c1.w, hi);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo[e] = hmul2(lo[e], sc[0][j >> 1]);
        hi[e] = hmul2(hi[e], sc[1][j >> 1]);
      }
      const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (j == 0)
          mma_f16_first(acc[n], a0, b[n].x, b[n].y);
        else
          mma_f16(acc[n], a0, b[n].x, b[n].y);
        mma_f16(acc[n], a1, b[n].z, b[n].w);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // a token without a place meets another's factor, and sums of zeros
      const float2 mul = NT > 1 || tok_p > 1 ? *reinterpret_cast<const float2*>(m + 8 * n) : make_float2(*m, 0.f);
      tot[n][0] = fmaf(acc[n][0], mul.x, tot[n][0]);
      tot[n][1] = fmaf(acc[n][1], mul.y, tot[n][1]);
      tot[n][2] = fmaf(acc[n][2], mul.x, tot[n][2]);
      tot[n][3] = fmaf(acc[n][3], mul.y, tot[n][3]);
    }
  };

#pragma unroll 1
  for (int st = 0; stage_lo(st) < p_hi; ++st) {
    if (st > 0) __syncthreads();
    stage_tokens(st);
    __syncthreads();
    const int n = share_n(st), lo = stage_lo(st) + share_lo(st);
    // batches of whole pieces, then what is left
    const int whole = max(0, min(n, a.k / kPiece - lo)) / kBatch * kBatch;
#pragma unroll 1
    for (int tile = 0; tile < (n > 0 ? n_tiles : 0); ++tile) {
      // rows past the CTA's last read that one's weights; their sums are not kept
      const int r = 16 * (tile0 + tile) + g;
      const uint8_t* code[2];
      const uint8_t* scale[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t row = static_cast<int64_t>(grp) * a.n + row0 + min(r + 8 * h, rows_cta - 1);
        code[h] = a.codes + row * code_row + static_cast<int64_t>(lo) * (kPiece / 2) + 16 * t;
        scale[h] = a.scales + row * scale_row + static_cast<int64_t>(lo) * (kPiece / 16) + 2 * t;
      }
      const uint8_t* x = smem + (kCodes ? share_lo(st) * kPiece + (x_here ? g : 0) * raw_pitch + 32 * t
                                        : 16 * (share_lo(st) * (NT * 4 * ru) + (x_here ? lane : 0)));
      const float* m = s_mul + share_lo(st) * tok_p + (y_here ? 2 * t : 0);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) tot[i][e] = 0.f;
      int p = 0;
      Weights w[kBatch];
      auto load = [&](int i, int ahead) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w[i].code[h] = load_stream(code[h] + (ahead + i) * (kPiece / 2));
          w[i].scale[h] = load_two(scale[h] + (ahead + i) * (kPiece / 16));
        }
      };
      if (kAhead && whole > 0)
#pragma unroll
        for (int i = 0; i < kBatch; ++i) load(i, 0);
#pragma unroll 1
      for (; p < whole; p += kBatch) {
        if (!kAhead)
#pragma unroll
          for (int i = 0; i < kBatch; ++i) load(i, 0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          add_piece(w[i], x + i * x_step, m + i * tok_p);
          if (kAhead && p + kBatch < whole) load(i, kBatch);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          code[h] += kBatch * (kPiece / 2);
          scale[h] += kBatch * (kPiece / 16);
        }
        x += kBatch * x_step;
        m += kBatch * tok_p;
      }
#pragma unroll 1
      for (; p < n; p += kBatch) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const bool here = p + i < n && static_cast<int64_t>(lo + p + i) * kPiece + 32 * t < a.k;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            w[i].code[h] = make_uint4(0, 0, 0, 0);
            w[i].scale[h] = 0;
            if (here) {
              w[i].code[h] = load_stream(code[h] + i * (kPiece / 2));
              w[i].scale[h] = load_two(scale[h] + i * (kPiece / 16));
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (i == 0 || p + i < n) add_piece(w[i], x + i * x_step, m + i * tok_p);  // uniform over the warp
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          code[h] += kBatch * (kPiece / 2);
          scale[h] += kBatch * (kPiece / 16);
        }
        x += kBatch * x_step;
        m += kBatch * tok_p;
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = 8 * i + 2 * t + (e & 1), at = r + 8 * (e >> 1);
          if (tok < tok_p && at < rows_cta) s_sum[(w_k * tok_p + tok) * pitch + at] += tot[i][e];
        }
    }
  }

  // ---- sums of the warps along k, then of the cluster's CTAs, each in its order
  if (wk > 1) {
    __syncthreads();
    for (int i = threadIdx.x; i < toks * pitch; i += kThreads) {
      float y = s_sum[i];
      for (int k = 1; k < wk; ++k) y += s_sum[k * tok_p * pitch + i];
      s_sum[i] = y;
    }
  }
  if (a.splits > 1)
    cluster_sync_all();
  else
    __syncthreads();
  const float factor = a.weight_scale != nullptr ? a.weight_scale[grp] : 1.f;
  const int each = (rows_cta + a.splits - 1) / a.splits;  // rows that a CTA finishes
  const int r_lo = min(split * each, rows_cta), r_n = min(each, rows_cta - r_lo);
  for (int i = threadIdx.x; i < r_n * toks; i += kThreads) {
    const int tok = i / r_n, r = r_lo + (i - tok * r_n);
    const float* const p = s_sum + tok * pitch + r;
    float y;
    if (a.splits > 1) {
      float v[kMaxSplits];
#pragma unroll
      for (int c = 0; c < kMaxSplits; ++c) v[c] = c < a.splits ? cluster_read(p, c) : 0.f;
      y = v[0];
#pragma unroll
      for (int c = 1; c < kMaxSplits; ++c) y += v[c];
    } else {
      y = *p;
    }
    y *= factor;
    const int64_t at = (tok0 + tok) * a.out_token + grp * a.out_group + row0 + r;
    if (a.out_float)
      static_cast<float*>(a.out)[at] = y;
    else
      static_cast<uint16_t*>(a.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
  }
  if (a.splits > 1) cluster_sync_all();  // nobody leaves while its sums are read
}

template <int NT, bool kCodes>
cudaError_t launch(const MatvecArgs& a, cudaStream_t stream) {
  const void* kernel = reinterpret_cast<const void*>(fp4_matvec_kernel<NT, kCodes>);
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = set_smem_limit_once(kernel, kSmemBytes, &configured);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (a.n + a.rows - 1) / a.rows * a.splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(a.groups),
                     static_cast<unsigned>((a.tokens + 8 * NT - 1) / (8 * NT)));
  cfg.blockDim = dim3(32 << warp_bits(NT));
  cfg.dynamicSmemBytes = static_cast<size_t>(a.smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(a.splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  MatvecArgs args = a;
  void* params[] = {&args};
  e = cudaLaunchKernelExC(&cfg, kernel, params);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// How the rows and k are split: modelled cycles of an SM whose CTAs are resident at
// once.  The longer of its pieces (`cycles` each with every warp busy) and of one
// warp's batches (`wait` each), the rounds in which the tokens are laid out, and
// what a cluster costs.  Clusters do not find a place on every SM (a group of SMs
// that share one has 18 to 20): a grid for all 152 ran in two rounds, so one SM in
// 19 is left out, and 5 in 19 where 8 CTAs have an SM each (32 bf16 tokens x 6144 x 6144
// 35.6 us with 18 such clusters, 20.5 with 14).  Measured, the chosen one first (row
// warps, splits, CTAs an SM): one token x 12288 x 6144 14.5 us with 2, 1, 3, then 14.7
// (8, 4, 3), 15.1 (4, 2, 3), 16.4 (1, 1, 3); 32 x 6144 x 12288 28.8 with 4, 4, 1, then 29.5
// (16, 4, 1), 31.7 (16, 8, 1), 35.0 (8, 2, 1); 8 x 8192 x 8192 19.2 with 2, 4, 3, where
// 8, 4, 3 takes 18.0.
bool plan(MatvecArgs* a, int nt, int tok_p) {
  const int per_piece = a->x_codes ? raw_piece_bytes(tok_p) : piece_bytes(nt, tok_p);
  const int pad = a->x_codes ? tok_p * kRawPad : 0;
  const int cycles = nt == 1 ? 64 : nt == 2 ? 100 : 170;
  const int wait = nt == 1 ? 4000 : nt == 2 ? 5500 : 4500;
  const int warps = 1 << warp_bits(nt);
  const int64_t all_sms = device_sm_count();
  const int pieces = (a->k + kPiece - 1) / kPiece;
  const int64_t others = static_cast<int64_t>(a->groups) * ((a->tokens + 8 * nt - 1) / (8 * nt));
  int64_t best = -1;
  for (int s = 1; s <= kMaxSplits && s <= pieces; s *= 2) {
    for (int res = resident(nt); res >= 1; --res) {
      const int64_t sms = s == 1 ? all_sms : all_sms * (s == 8 && res == 1 ? 14 : 18) / 19;
      int64_t blocks = sms * res / (s * others);
      if (blocks < 1) blocks = 1;
      if (blocks > a->n) blocks = a->n;
      int64_t rows = (a->n + blocks - 1) / blocks;
      if (rows > kMaxRows) rows = kMaxRows;
      const int slice = (pieces + s - 1) / s;
      int most = a->x_codes ? (kSmemBytes / res - 2048 - pad) * 3 / 4 / per_piece : stage_tasks(nt) / tok_p;
      if (most < 1) continue;
      const int stage = slice < most ? slice : most;
      // many rows and tokens: as many rows as leave their sums room beside a stage, in rounds
      const int64_t room = kSmemBytes / res - (res > 1 ? 1024 : 0) - static_cast<int64_t>(stage) * per_piece - pad;
      const int64_t fit = (room / (4 * tok_p) - 4) / 16 * 16;
      if (fit < 16) continue;
      if (rows > fit) rows = fit;
      const int tiles = static_cast<int>((rows + 15) / 16);
      const int64_t rounds = ((a->n + rows - 1) / rows * s * others + sms * res - 1) / (sms * res);
      const int stages = (slice + stage - 1) / stage;
      const int lays = a->x_codes ? stages : (stage * tok_p + warps * 16 - 1) / (warps * 16) * stages;
      for (int bits = warp_bits(nt); bits >= 0; --bits) {
        const int wr = 1 << bits, wk = warps / wr;
        const int64_t smem = static_cast<int64_t>(stage) * per_piece + pad + sum_bytes(tok_p, wk, rows);
        if (smem - static_cast<int64_t>(stage) * per_piece - pad > room) continue;
        const int share = (stage + wk - 1) / wk;
        const int64_t batches = static_cast<int64_t>(stages) * ((tiles + wr - 1) / wr) *
                                ((share + batch(nt) - 1) / batch(nt));
        const int64_t work = static_cast<int64_t>(res) * tiles * slice * cycles;
        const int64_t cost =
            rounds * ((work > batches * wait ? work : batches * wait) + lays * 4000 + (s > 1 ? 3500 + 500 * s : 0));
        if (best < 0 || cost < best) {
          best = cost;
          a->row_warps_bits = bits;
          a->slice = slice;
          a->splits = s;
          a->rows = static_cast<int>(rows);
          a->stage = stage;
          a->smem = static_cast<int>(smem);
        }
      }
    }
  }
  return best >= 0;
}

}  // namespace

cudaError_t launch_fp4_matvec(MatvecArgs a, cudaStream_t stream) {
  const int nt = a.tokens <= 8 ? 1 : a.tokens <= 16 ? 2 : 4;
  int tok_p = 8 * nt;
  while (nt == 1 && tok_p / 2 >= a.tokens) tok_p /= 2;
  if (!plan(&a, nt, tok_p)) return cudaErrorInvalidConfiguration;
  if (a.x_codes) {
    if (nt == 1) return launch<1, true>(a, stream);
    if (nt == 2) return launch<2, true>(a, stream);
    return launch<4, true>(a, stream);
  }
  if (nt == 1) return launch<1, false>(a, stream);
  if (nt == 2) return launch<2, false>(a, stream);
  return launch<4, false>(a, stream);
}

}  // namespace mla
