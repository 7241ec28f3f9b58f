// The residual's addition, the norm behind it and its output in 8 bits.
//
// Per row of D values:  h = x + r,  y = h / sqrt(mean(h^2) + eps) * w, and for
// each group of 128 values (or the row)  s = max|y| / 448,  code = e4m3(y / s).
// Float throughout: h is rounded only where it is stored (to the residual's
// type), y only to its code, so the norm sees the sum before that rounding.
//
// Split.  A team of 1 to 16 warps has a row; lane l of the team has the 8-value
// chunks l, l + 32 W, ...: loads are whole 16-byte accesses of neighbouring
// lanes, and a group of 128 is half a warp's share of one load, so that its
// largest value needs four shuffles.  Teams walk the rows with a stride, twice as
// many CTAs as are resident.  Holding the next row's values in registers while one
// is worked on costs more warps than it hides: 24,000 rows of 6144 with a bf16
// residual took 175 us (a team of 4 warps with 6 chunks a lane 205), then 160
// without it, and 155 with the larger grid (one CTA for every row 155).
//
// Bound: HBM, there 1,037 MB in 155 us: 6,690 GB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

enum Residual { kNone = 0, kBf16 = 1, kFloat = 2 };

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// W warps a row, C chunks a lane.
template <int W, int C, int R>
__global__ void __launch_bounds__(W > 8 ? 32 * W : 256) add_norm_quant_kernel(const AddNormArgs a) {
  constexpr int kWarps = W > 8 ? W : 8;
  constexpr int kTeams = kWarps / W;
  constexpr int kLanes = 32 * W;
  constexpr int kRes = R == kFloat ? 2 : R == kBf16 ? 1 : 0;  // 16-byte loads of the residual a chunk
  __shared__ float s_sum[2][kWarps];
  __shared__ uint32_t s_max[2][kWarps];
  // Plain loads from here on: the grid may be resident before its inputs are written.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int team = threadIdx.x / kLanes, tl = threadIdx.x % kLanes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = a.dim / 8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kTeams;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + team;

  uint4 nx[C], nr[C][kRes > 0 ? kRes : 1];
  auto load = [&] {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = tl + c * kLanes;
      if (i < chunks) {
        nx[c] = reinterpret_cast<const uint4*>(a.x + row * a.x_stride)[i];
        if constexpr (R == kBf16)
          nr[c][0] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.residual) + row * a.res_stride)[i];
        if constexpr (R == kFloat) {
          const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(a.residual) + row * a.res_stride) + 2 * i;
          nr[c][0] = p[0];
          nr[c][1] = p[1];
        }
      } else {
        nx[c] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < kRes; ++k) nr[c][k] = make_uint4(0, 0, 0, 0);
      }
    }
  };
  // Over the team's lanes, the same in each of them.  The warps' parts stand in
  // shared memory; `turn` alternates, so one barrier a reduction is enough.
  int turn = 0;
  auto team_barrier = [&] { named_bar_sync(1 + team, kLanes); };
  auto team_sum = [&](float v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
    if constexpr (W > 1) {
      if (lane == 0) s_sum[turn][warp] = v;
      team_barrier();
      v = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) v += s_sum[turn][team * W + k];
      turn ^= 1;
    }
    return v;
  };
  // Magnitudes as integers: a NaN is larger than every value and stays.
  auto team_max = [&](uint32_t v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, m));
    if constexpr (W > 1) {
      if (lane == 0) s_max[turn][warp] = v;
      team_barrier();
      v = 0;
#pragma unroll
      for (int k = 0; k < W; ++k) v = max(v, s_max[turn][team * W + k]);
      turn ^= 1;
    }
    return v;
  };

#pragma unroll 1
  for (; row < a.tokens; row += stride) {
    load();
    float h[C][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      unpack8(nx[c], h[c]);
      float r[8];
      if constexpr (R == kBf16) unpack8(nr[c][0], r);
      if constexpr (R == kFloat) {
        const uint32_t w[8] = {nr[c][0].x, nr[c][0].y, nr[c][0].z, nr[c][0].w, nr[c][1].x, nr[c][1].y, nr[c][1].z, nr[c][1].w};
#pragma unroll
        for (int k = 0; k < 8; ++k) r[k] = __uint_as_float(w[k]);
      }
      if constexpr (R != kNone) {
#pragma unroll
        for (int k = 0; k < 8; ++k) h[c][k] += r[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(h[c][k], h[c][k], ss);
    }
    if constexpr (R != kNone) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int i = tl + c * kLanes;
        if (i >= chunks) continue;
        if constexpr (R == kBf16) {
          reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.residual_out) + row * a.res_out_stride)[i] =
              make_uint4(bf16x2_rn(h[c][0], h[c][1]), bf16x2_rn(h[c][2], h[c][3]), bf16x2_rn(h[c][4], h[c][5]),
                         bf16x2_rn(h[c][6], h[c][7]));
        } else {
          float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.residual_out) + row * a.res_out_stride) + 2 * i;
          p[0] = make_float4(h[c][0], h[c][1], h[c][2], h[c][3]);
          p[1] = make_float4(h[c][4], h[c][5], h[c][6], h[c][7]);
        }
      }
    }
    ss = team_sum(ss);
    float mean = ss * a.inv_dim + a.eps, down = 1.f;
    if (mean == INFINITY) {
      // squares, or the largest eps with them, past float's range: with values 2^-80 as large
      // they add up to less than 2^110 (a row that holds an infinity stays as it is)
      constexpr float kDown = 8.271806125530277e-25f;  // 2^-80
      float small = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float v = h[c][k] * kDown;
          small = fmaf(v, v, small);
        }
      mean = fmaf(team_sum(small), a.inv_dim, a.eps * kDown * kDown);
      down = kDown;
    }
    // The quotients do not depend on the row's factor: the values are scaled by its power of
    // two alone, which rounds nothing, and the rest of it meets the stored scales.
    float rstd = rsqrtf(mean), rest = 1.f;
    if (mean < INFINITY) {
      rest = __int_as_float((__float_as_int(rstd) & 0x007FFFFF) | 0x3F800000);
      rstd = __int_as_float(__float_as_int(rstd) & 0x7F800000) * down;
    }
    uint32_t mx[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = tl + c * kLanes;
      float w[8];
      unpack8(i < chunks ? reinterpret_cast<const uint4*>(a.weight)[i] : make_uint4(0, 0, 0, 0), w);
      mx[c] = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        h[c][k] = i < chunks ? h[c][k] * rstd * w[k] : 0.f;
        mx[c] = max(mx[c], __float_as_uint(h[c][k]) & 0x7FFFFFFFu);
      }
    }
    if (a.group == 0) {
#pragma unroll
      for (int c = 1; c < C; ++c) mx[0] = max(mx[0], mx[c]);
      mx[0] = team_max(mx[0]);
#pragma unroll
      for (int c = 1; c < C; ++c) mx[c] = mx[0];
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int m = 8; m > 0; m >>= 1) mx[c] = max(mx[c], __shfl_xor_sync(0xFFFFFFFFu, mx[c], m));
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = tl + c * kLanes;
      if (i >= chunks) continue;
      const float s = __fdiv_rn(__uint_as_float(mx[c]), 448.f);
      float q[8];
      if (s >= 1.17549435e-38f && s < INFINITY) {
        const float r = __frcp_rn(s);
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = div_rn(h[c][k], s, r);
      } else {  // nothing but zeros, a reciprocal past float's range, or no number
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = s == 0.f ? 0.f : __fdiv_rn(h[c][k], s);
      }
      const uint32_t lo = f32x2_to_e4m3x2(q[1], q[0]) | (f32x2_to_e4m3x2(q[3], q[2]) << 16);
      const uint32_t hi = f32x2_to_e4m3x2(q[5], q[4]) | (f32x2_to_e4m3x2(q[7], q[6]) << 16);
      reinterpret_cast<uint2*>(a.codes + row * a.dim)[i] = make_uint2(lo, hi);
      if (a.group == 0 ? i == 0 : (i & 15) == 0) a.scales[row * a.scale_groups + (a.group == 0 ? 0 : i >> 4)] = s * rest;
    }
  }
}

template <int W, int C>
cudaError_t launch(const AddNormArgs& a, cudaStream_t stream) {
  constexpr int kWarps = W > 8 ? W : 8;
  constexpr int kTeams = kWarps / W;
  const int64_t need = (a.tokens + kTeams - 1) / kTeams;
  const int64_t room = static_cast<int64_t>(device_sm_count()) * (W > 8 ? 4 : 8);
  const unsigned grid = static_cast<unsigned>(need < room ? need : room);
  const void* kernel = a.residual_type == kNone   ? reinterpret_cast<const void*>(add_norm_quant_kernel<W, C, kNone>)
                       : a.residual_type == kBf16 ? reinterpret_cast<const void*>(add_norm_quant_kernel<W, C, kBf16>)
                                                  : reinterpret_cast<const void*>(add_norm_quant_kernel<W, C, kFloat>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  AddNormArgs args = a;
  void* params[] = {&args};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, params);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_norm_quant(const AddNormArgs& a, cudaStream_t stream) {
  const int chunks = a.dim / 8;
  if (chunks <= 32) return launch<1, 1>(a, stream);
  if (chunks <= 64) return launch<1, 2>(a, stream);
  if (chunks <= 128) return launch<2, 2>(a, stream);
  if (chunks <= 256) return launch<4, 2>(a, stream);
  if (chunks <= 512) return launch<8, 2>(a, stream);
  if (chunks <= 768) return launch<8, 3>(a, stream);
  if (chunks <= 1024) return launch<16, 2>(a, stream);
  return launch<16, 4>(a, stream);
}

}  // namespace mla
