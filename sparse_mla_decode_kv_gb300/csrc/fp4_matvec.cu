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
// Split.  A warp has 16 MT rows of weights as the A operand and 8 NT tokens as
// B (m16n8k16).  Which 16 values of k an MMA adds up is free as long as both
// operands agree: lane t of a row's four has the 32 consecutive codes 32 t ..
// of each 128, so a lane's codes are one 16-byte load, its scales one 2-byte
// load, and every group's scale is needed by one lane only.  The tokens are laid
// out in shared memory in the order in which the lanes read them.  A CTA is WR x
// WK warps: rows, and 128-value pieces of k in turn; up to 8 CTAs of a cluster
// have slices of k.  Their sums are joined in shared memory in one order, so a
// call gives the same bits every time.
//
// Bound: HBM, 9/16 byte a weight.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kPiece = 128;  // values of k per step of a warp
// Tokens' values of one piece, in units of 8: [n-tile][4][8 tokens x 4 lanes],
// the four 34 units apart so that a token's sixteen units fall into different banks
// when they are written.
constexpr int kUnitStride = 34;
constexpr int kPieceUnits = 4 * kUnitStride;

__host__ __device__ constexpr int depth(int nt) { return nt == 1 ? 4 : 2; }  // pieces on their way in registers
__host__ __device__ constexpr int stage_pieces(int nt) { return nt == 1 ? 32 : nt == 2 ? 16 : 8; }
__host__ __device__ constexpr int piece_bytes(int nt) { return nt * (kPieceUnits * 16 + 8 * 4); }
// Joined sums: [WK][tokens][rows + 4] floats over the place of the tokens.
__host__ __device__ constexpr int sum_bytes(int mt, int nt) { return 8 * nt * (16 * mt + 4) * kWarps * 4; }
__host__ __device__ constexpr int smem_bytes(int mt, int nt) {
  const int a = stage_pieces(nt) * piece_bytes(nt), b = sum_bytes(mt, nt);
  return a > b ? a : b;
}

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

template <int MT, int NT, bool kCodes>
__global__ void __launch_bounds__(kThreads, 2) fp4_matvec_kernel(const MatvecArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* const s_x = reinterpret_cast<uint4*>(smem);
  float* const s_mul = reinterpret_cast<float*>(smem + stage_pieces(NT) * NT * kPieceUnits * 16);
  constexpr int kTokens = 8 * NT;
  constexpr int kDepth = depth(NT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int wr = a.row_warps, wk = kWarps / wr;
  const int split = blockIdx.x % a.splits;
  const int rows_cta = 16 * MT * wr;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / a.splits) * rows_cta;
  const int grp = blockIdx.y;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.z) * kTokens;
  const int toks = static_cast<int>(min(static_cast<int64_t>(kTokens), a.tokens - tok0));
  const int pieces = (a.k + kPiece - 1) / kPiece;
  const int p0 = static_cast<int>(static_cast<int64_t>(pieces) * split / a.splits);
  const int p1 = static_cast<int>(static_cast<int64_t>(pieces) * (split + 1) / a.splits);
  const int w_row = warp % wr, w_k = warp / wr;
  const int steps = (p1 - p0 + wk - 1) / wk;               // of every warp
  const int stage_steps = stage_pieces(NT) / wk;           // of every warp with the same tokens in shared memory

  // rows past the last read the last one's weights, their sums are not written
  const uint8_t* code[MT][2];
  const uint8_t* scale[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t r = min(row0 + 16 * (MT * w_row + m) + 8 * h + g, static_cast<int64_t>(a.n) - 1);
      const int64_t at = static_cast<int64_t>(grp) * a.n + r;
      code[m][h] = a.codes + at * (a.k / 2) + 16 * t;
      scale[m][h] = a.scales + at * (a.k / 16) + 2 * t;
    }
  Weights buf[kDepth][MT];
  auto fetch = [&](int step, Weights (&w)[MT]) {
    const int p = p0 + w_k + wk * step;
    const bool here = p < p1 && p * kPiece + 32 * t < a.k;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w[m].code[h] = here ? load_stream(code[m][h] + static_cast<int64_t>(p) * (kPiece / 2)) : make_uint4(0, 0, 0, 0);
        w[m].scale[h] = here ? *reinterpret_cast<const unsigned short*>(scale[m][h] + static_cast<int64_t>(p) * (kPiece / 16)) : 0;
      }
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) fetch(i, buf[i]);

  // The tokens of pieces [p0 + at, ...): half a warp has one token's piece, 8
  // values a lane.
  auto stage = [&](int at) {
    const int count = min(stage_pieces(NT), p1 - p0 - at);
    const int u = lane & 15;
    const uint32_t half = lane & 16 ? 0xFFFF0000u : 0x0000FFFFu;  // the halves go round a different number of times
    for (int i = threadIdx.x >> 4; i < count * toks; i += kThreads / 16) {
      const int piece = i / toks, tok = i - piece * toks;
      const int k0 = (p0 + at + piece) * kPiece + 8 * u;
      const int64_t off = (tok0 + tok) * a.x_token + grp * a.x_group + k0;
      uint32_t h[4] = {0, 0, 0, 0};
      float mul = 1.f;
      if constexpr (kCodes) {
        if (k0 < a.k) {
          const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) + off);
          uint32_t lo[2], hi[2];
          e4m3x4_to_f16x2x2(v.x, lo);
          e4m3x4_to_f16x2x2(v.y, hi);
          h[0] = lo[0];
          h[1] = lo[1];
          h[2] = hi[0];
          h[3] = hi[1];
        }
        if (u == 0) mul = a.x_scales[((tok0 + tok) * a.groups + grp) * a.x_scale_groups + (a.x_scale_groups > 1 ? p0 + at + piece : 0)];
      } else {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (k0 < a.k) v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + off);
        uint32_t mx = bf16x8_absmax_bits(v);
#pragma unroll
        for (int m = 8; m > 0; m >>= 1) mx = max(mx, __shfl_xor_sync(half, mx, m));
        const int shift = query_shift(mx);
        const float up = pow2f(shift);
        mul = pow2f(-shift);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half2 p = __floats2half2_rn(bf16_bits_to_f32(w[j] & 0xFFFFu) * up, bf16_bits_to_f32(w[j] >> 16) * up);
          h[j] = *reinterpret_cast<const uint32_t*>(&p);
        }
      }
      const int nt = tok >> 3;
      s_x[(piece * NT + nt) * kPieceUnits + (u & 3) * kUnitStride + (tok & 7) * 4 + (u >> 2)] = make_uint4(h[0], h[1], h[2], h[3]);
      if (u == 0) s_mul[piece * kTokens + tok] = mul;
    }
  };

  if (toks < kTokens) {  // the tokens that are not there are zeros
    for (int i = threadIdx.x; i < stage_pieces(NT) * piece_bytes(NT) / 16; i += kThreads) s_x[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  float tot[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) tot[m][n][i] = 0.f;

#pragma unroll 1
  for (int s0 = 0; s0 < steps; s0 += kDepth) {
    if (s0 % stage_steps == 0) {
      if (s0 > 0) __syncthreads();
      stage(s0 * wk);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      const int step = s0 + i;
      if (step >= steps) break;
      const int local = (step % stage_steps) * wk + w_k;
      const bool here = p0 + w_k + wk * step < p1;  // uniform over the warp
      if (here) {
        float acc[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][n][e] = 0.f;
        uint32_t sc[MT][2][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t two = buf[i][m].scale[h];
            sc[m][h][0] = e4m3x2_to_f16x2((two & 0xFFu) * 0x0101u);
            sc[m][h][1] = e4m3x2_to_f16x2((two >> 8) * 0x0101u);
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 b[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) b[n] = s_x[(local * NT + n) * kPieceUnits + j * kUnitStride + lane];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint4 c0 = buf[i][m].code[0], c1 = buf[i][m].code[1];
            uint32_t lo[4], hi[4];
            e2m1x8_to_f16x2x4(j == 0 ? c0.x : j == 1 ? c0.y : j == 2 ? c0.z : c0.w, lo);
            e2m1x8_to_f16x2x4(j == 0 ? c1.x : j == 1 ? c1.y : j == 2 ? c1.z : c1.w, hi);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              lo[e] = hmul2(lo[e], sc[m][0][j >> 1]);
              hi[e] = hmul2(hi[e], sc[m][1][j >> 1]);
            }
            const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_f16(acc[m][n], a0, b[n].x, b[n].y);
              mma_f16(acc[m][n], a1, b[n].z, b[n].w);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float2 mul = *reinterpret_cast<const float2*>(s_mul + local * kTokens + 8 * n + 2 * t);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            tot[m][n][0] = fmaf(acc[m][n][0], mul.x, tot[m][n][0]);
            tot[m][n][1] = fmaf(acc[m][n][1], mul.y, tot[m][n][1]);
            tot[m][n][2] = fmaf(acc[m][n][2], mul.x, tot[m][n][2]);
            tot[m][n][3] = fmaf(acc[m][n][3], mul.y, tot[m][n][3]);
          }
        }
      }
      fetch(step + kDepth, buf[i]);
    }
  }

  // ---- sums of the warps along k, then of the cluster's CTAs, each in its order
  __syncthreads();
  float* const s_sum = reinterpret_cast<float*>(smem);  // [w_k][token][row]
  const int pitch = rows_cta + 4;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s_sum[(w_k * kTokens + 8 * n + 2 * t + (e & 1)) * pitch + 16 * (MT * w_row + m) + g + 8 * (e >> 1)] = tot[m][n][e];
  if (a.splits > 1)
    cluster_sync_all();
  else
    __syncthreads();
  const float factor = a.weight_scale != nullptr ? a.weight_scale[grp] : 1.f;
  const int each = rows_cta / a.splits;  // rows that this CTA finishes, and the remainder in the last
  const int r_lo = split * each, r_n = split + 1 == a.splits ? rows_cta - r_lo : each;
  for (int i = threadIdx.x; i < r_n * toks; i += kThreads) {
    const int tok = i / r_n, r = r_lo + (i - tok * r_n);
    if (row0 + r >= a.n) continue;
    float y = 0.f;
    for (int c = 0; c < a.splits; ++c) {
      for (int k = 0; k < wk; ++k) {
        const float* p = s_sum + (k * kTokens + tok) * pitch + r;
        y += a.splits > 1 ? cluster_read(p, c) : *p;
      }
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

template <int MT, int NT, bool kCodes>
cudaError_t launch(const MatvecArgs& a, cudaStream_t stream) {
  const void* kernel = reinterpret_cast<const void*>(fp4_matvec_kernel<MT, NT, kCodes>);
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = set_smem_limit_once(kernel, smem_bytes(MT, NT), &configured);
  if (e != cudaSuccess) return e;
  const int64_t rows = 16LL * MT * a.row_warps;
  const int64_t blocks = (a.n + rows - 1) / rows * a.splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(a.groups),
                     static_cast<unsigned>((a.tokens + 8 * NT - 1) / (8 * NT)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(MT, NT);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(a.splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  MatvecArgs args = a;
  void* params[] = {&args};
  e = cudaLaunchKernelExC(&cfg, kernel, params);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp4_matvec(MatvecArgs a, cudaStream_t stream) {
  const int nt = a.tokens <= 8 ? 1 : a.tokens <= 16 ? 2 : 4;
  const int mt = nt == 2 ? 2 : 1;
  const int64_t sms = device_sm_count();
  const int pieces = (a.k + kPiece - 1) / kPiece;
  const int64_t others = static_cast<int64_t>(a.groups) * ((a.tokens + 8 * nt - 1) / (8 * nt));
  // Modelled time of the call: CTAs in waves of two a SM, each its pieces' weights and
  // tokens (in rows) and a start worth 2,000 row pieces.
  int64_t best = -1;
  for (int wr = nt == 4 ? 2 : 1; wr <= kWarps; wr *= 2)  // a stage is a whole number of every warp's register pieces
    for (int s = 1; s <= 8 && s <= pieces; ++s) {
      const int64_t rows = 16LL * mt * wr;
      const int64_t ctas = (a.n + rows - 1) / rows * s * others;
      const int64_t waves = (ctas + 2 * sms - 1) / (2 * sms);
      const int wk = kWarps / wr;
      const int64_t mine = ((pieces + s - 1) / s + wk - 1) / wk * wk;
      const int64_t cost = waves * (mine * (rows + 8 * nt) + 2000 + (s > 1 ? 500 : 0));
      if (best < 0 || cost < best) {
        best = cost;
        a.row_warps = wr;
        a.splits = s;
      }
    }
  if (a.x_codes) {
    if (nt == 1) return launch<1, 1, true>(a, stream);
    if (nt == 2) return launch<2, 2, true>(a, stream);
    return launch<1, 4, true>(a, stream);
  }
  if (nt == 1) return launch<1, 1, false>(a, stream);
  if (nt == 2) return launch<2, 2, false>(a, stream);
  return launch<1, 4, false>(a, stream);
}

}  // namespace mla
