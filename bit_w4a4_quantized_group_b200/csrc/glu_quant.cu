// Activation with an FP8 output (svdq_glu_quantize_act).
//
//   y_k = act(gate_k) [* up_k] [/ lambda_k],   codes = e4m3(y / 2^e), 2^e per 128 elements.
//
// Both activations have the form x * sigmoid(t) = x / (1 + exp(-t)): SiLU with t = x, the tanh
// form of GELU with t = 2 sqrt(2/pi) (x + 0.044715 x^3), since 1 + tanh(u) = 2 / (1 + exp(-2u)).
// This form has no cancellation for negative x, and its ends are right without a branch: exp
// overflows to infinity, whose reciprocal is 0, or underflows to 0 and leaves x.  exp and the
// reciprocal are the hardware's approximations (2 and 1 units in the last place); the divide by
// lambda shares the reciprocal, 1 / ((1 + exp(-t)) lambda).  All of it is far inside the E4M3 step of 2^-4.
// A reciprocal below 2^-126 becomes 0 before up multiplies it: the interface states that, since a form
// without it (the exponential halved and applied twice) would cost every element two more operations.
//
// What bounds it: memory (3 bytes per element, 5 with gating).  Eight lanes hold a group: a
// thread has two 16-byte chunks of it (64 elements apart, so that the lanes of a load are
// neighbours) in each of kRows rows, all its loads in flight together.  The exponentials and
// reciprocals (two per element, 16 a clock and SM) and the instruction issue are each busy about as
// long as memory, so products run on pairs (f32x2), row overheads are spread over 16 elements, and
// large ungated calls fetch a thread's next rows under the stores of the current ones.  Two elements
// share a reciprocal in gated calls without lambda (SiLU 2304 x 12288, rows x K: 22.9 us against 24.5); without
// gating the branch costs more than it saves (GELU 4608 x 12288: 38.6 us against 34.1), and with lambda the products
// may leave the range.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "fp8_quant.cuh"
#include "ptx.cuh"
#include "svdq.h"
#include "svdq_device.cuh"

namespace svdq {
namespace {

constexpr int kThreads = 128;
constexpr int kGroups = kThreads / 8;          // 128-element groups across a CTA
constexpr int kRows = 2;
constexpr int kIters = 4;

// -t log2(e) of a pair: the factor -log2(e) is folded into the constants, so that exp(-t) is one ex2.
template <int ACT>
__device__ __forceinline__ float2 neg_t_log2(float2 x) {
  constexpr float kLog2e = 1.4426950408889634f, kC1 = -2.f * 0.7978845608028654f * kLog2e, kC3 = kC1 * 0.044715f;
  if (ACT == SVDQ_ACT_SILU) return __fmul2_rn(x, make_float2(-kLog2e, -kLog2e));
  return __fmul2_rn(x, __ffma2_rn(__fmul2_rn(x, x), make_float2(kC3, kC3), make_float2(kC1, kC1)));
}
__device__ __forceinline__ float ex2_approx(float t) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return e;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {      // NaN if one of them is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// d = 1 / d for 8 elements.  PAIRED (all d >= 1 or NaN): 1 / (a b) once, times b and times a, where every
// product is in range; a NaN or an exp beyond 2^100 among the eight takes the plain way, each by itself.
template <bool PAIRED>
__device__ __forceinline__ void reciprocals(float2 (&d)[4]) {
  float m = 0.f;
  float p[4];
  if (PAIRED) {
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = d[e].x * d[e].y;
    m = max_nan(max_nan(p[0], p[1]), max_nan(p[2], p[3]));
  }
  if (PAIRED && m < 0x1p100f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float r = rcp_approx(p[e]);
      d[e] = make_float2(r * d[e].y, r * d[e].x);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = make_float2(rcp_approx(d[e].x), rcp_approx(d[e].y));
  }
}

// ITERS row pairs per CTA, one after the other, the next pair's loads under the current one's stores.
template <int ACT, bool GATED, bool LAM, int ITERS>
__global__ void __launch_bounds__(kThreads) glu_quant_kernel(GluParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int t = static_cast<int>(threadIdx.x);
  const int G = p.K >> 7;
  const int cblocks = (G + kGroups - 1) / kGroups;
  const int row0 = static_cast<int>(blockIdx.x / static_cast<unsigned>(cblocks)) * (kRows * ITERS);
  const int grp = static_cast<int>(blockIdx.x % static_cast<unsigned>(cblocks)) * kGroups + (t >> 3);
  if (row0 >= p.M) {      // the CTA behind the last row block
    fp8_zero_padding(p.scales, p.M, p.K, p.sfb, t, kThreads);
    return;
  }
  const bool on = grp < G;
  const int row_end = min(p.M, row0 + kRows * ITERS);
  const size_t col = static_cast<size_t>(grp) * 128 + (t & 7) * 8;     // and col + 64
  const int nsc = grp == G - 1 ? 4 * p.sfb - grp : 1;                  // scale bytes that its lanes write
  uint4 g[kRows][2], u[GATED ? kRows : 1][2];
  auto load = [&](int r) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const bool in = on && r + i < row_end;
      const __nv_bfloat16* src = p.gate + static_cast<size_t>(r + i) * p.ldg + col;
#pragma unroll
      for (int h = 0; h < 2; ++h) g[i][h] = in ? ld_global_v4_na(src + 64 * h) : make_uint4(0, 0, 0, 0);
      if (GATED) {
        const __nv_bfloat16* srcu = p.up + static_cast<size_t>(r + i) * p.ldu + col;
#pragma unroll
        for (int h = 0; h < 2; ++h) u[i][h] = in ? ld_global_v4_na(srcu + 64 * h) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  load(row0);
#pragma unroll 1
  for (int r = row0; r < row_end; r += kRows) {
    const int rows = min(kRows, row_end - r);
    // y of every row, and the scale byte that this thread's own elements need.  The byte grows with the
    // absolute value, so the group's byte is the largest of its lanes': two rows' bytes go through one
    // shuffle as 16-bit halves.
    float2 y[kRows][2][4];
    float amax[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) amax[i] = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float2 lam[4];
      if (LAM) {
        const float4* lp = reinterpret_cast<const float4*>(p.lam + (on ? col : 0) + 64 * h);
        const float4 l0 = __ldg(lp), l1 = __ldg(lp + 1);
        lam[0] = make_float2(l0.x, l0.y);
        lam[1] = make_float2(l0.z, l0.w);
        lam[2] = make_float2(l1.x, l1.y);
        lam[3] = make_float2(l1.z, l1.w);
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const uint32_t gx[4] = {g[i][h].x, g[i][h].y, g[i][h].z, g[i][h].w};
        float2 d[4];                                    // then its reciprocal
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 nt = neg_t_log2<ACT>(make_float2(bf16x2_lo(gx[e]), bf16x2_hi(gx[e])));
          d[e] = __fadd2_rn(make_float2(ex2_approx(nt.x), ex2_approx(nt.y)), make_float2(1.f, 1.f));
          if (LAM) d[e] = __fmul2_rn(d[e], lam[e]);     // one reciprocal serves both divides
        }
        reciprocals<GATED && !LAM>(d);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2 v = __fmul2_rn(make_float2(bf16x2_lo(gx[e]), bf16x2_hi(gx[e])), d[e]);
          if (GATED) {
            const uint32_t ux[4] = {u[i][h].x, u[i][h].y, u[i][h].z, u[i][h].w};
            v = __fmul2_rn(v, make_float2(bf16x2_lo(ux[e]), bf16x2_hi(ux[e])));
          }
          amax[i] = fmaxf(amax[i], fmaxf(fabsf(v.x), fabsf(v.y)));
          y[i][h][e] = v;
        }
      }
    }
    if (ITERS > 1) load(r + kRows);
    uint32_t sb[kRows / 2];
#pragma unroll
    for (int i = 0; i < kRows / 2; ++i) {
      sb[i] = fp8_scale_byte(amax[2 * i]) | (fp8_scale_byte(amax[2 * i + 1]) << 16);
#pragma unroll
      for (int o = 1; o <= 4; o <<= 1) sb[i] = max_u16x2(sb[i], __shfl_xor_sync(0xffffffffu, sb[i], o));
    }
    uint8_t* sc = p.scales + fp8_sf_offset(r, grp, p.sfb);      // r is even: the next row's is 16 bytes on
    uint8_t* dst = p.codes + static_cast<size_t>(r) * p.K + col;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (i >= rows || !on) break;
      const uint32_t b = (sb[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
      const float inv = fp8_inv_scale(b);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (SVDQ_IN_GLOBAL(col + 64 * h + 8 <= static_cast<size_t>(p.K), p.err))
          *reinterpret_cast<uint2*>(dst + 64 * h) = fp8_codes8(y[i][h], inv);
      }
      dst += p.K;
      // lane 0 has the group's byte; behind the row's last group the next lanes have the padding groups, up
      // to the next multiple of four, which is the same 4-byte word
      if ((t & 7) < nsc) sc[16 * i + (t & 7)] = (t & 7) == 0 ? static_cast<uint8_t>(b) : 0;
    }
  }
}

template <int ACT>
cudaError_t launch(const GluParams& p, int iters, const cudaLaunchConfig_t& cfg) {
  if (p.up) return p.lam ? cudaLaunchKernelEx(&cfg, glu_quant_kernel<ACT, true, true, 1>, p)
                         : cudaLaunchKernelEx(&cfg, glu_quant_kernel<ACT, true, false, 1>, p);
  if (iters > 1) return p.lam ? cudaLaunchKernelEx(&cfg, glu_quant_kernel<ACT, false, true, kIters>, p)
                              : cudaLaunchKernelEx(&cfg, glu_quant_kernel<ACT, false, false, kIters>, p);
  return p.lam ? cudaLaunchKernelEx(&cfg, glu_quant_kernel<ACT, false, true, 1>, p)
               : cudaLaunchKernelEx(&cfg, glu_quant_kernel<ACT, false, false, 1>, p);
}

}  // namespace

cudaError_t launch_glu_quant(const GluParams& p, cudaStream_t s, int* variant) {
  const int64_t cblocks = (p.K / 128 + kGroups - 1) / kGroups;
  // Four row pairs per CTA where that still leaves 3000 CTAs, four rounds of the device (GELU with lambda,
  // 4608 x 12288: 35.8 us against 37.6 with one and 37.2 with two; SiLU 8192 x 8192: 41.8 against 46.1;
  // 1000 rows of a small K get slower).  With gating a pair has twice the loads, and the next pair's
  // registers cost more than they give (SiLU with lambda, 8192 x 11008: 9% slower than the 74 us without).
  const int iters = !p.up && cblocks * ((static_cast<int64_t>(p.M) + 2 * kIters - 1) / (2 * kIters)) >= 3000 ? kIters : 1;
  *variant = iters;
  const int64_t rows = kRows * iters;
  const int64_t grid = cblocks * ((p.M + rows - 1) / rows) + (p.M % 128 ? 1 : 0);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = p.act == SVDQ_ACT_SILU ? launch<SVDQ_ACT_SILU>(p, iters, cfg) : launch<SVDQ_ACT_GELU_TANH>(p, iters, cfg);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace svdq
