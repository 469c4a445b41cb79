// Activation with an FP8 output (svdq_glu_quantize_act).
//
//   y_k = act(gate_k) [* up_k] [/ lambda_k],   codes = e4m3(y / 2^e), 2^e per 128 elements.
//
// Both activations have the form x * sigmoid(t) = x / (1 + exp(-t)): SiLU with t = x, the tanh
// form of GELU with t = 2 sqrt(2/pi) (x + 0.044715 x^3), since 1 + tanh(u) = 2 / (1 + exp(-2u)).
// This form has no cancellation for negative x, and its ends are right without a branch: exp
// overflows to infinity, whose reciprocal is 0, or underflows to 0 and leaves x.  exp and the
// reciprocal are the hardware's approximations (2 and 1 units in the last place); a divide by
// lambda is a product with its reciprocal.  All of it is far inside the E4M3 step of 2^-4.
//
// What bounds it: memory (3 bytes per element, 5 with gating).  A thread holds 8 elements (16
// bytes of each input) of kRows rows of the same columns, so that all its loads are in flight
// together and lambda is read once per kRows rows; 16 lanes hold a group.
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
constexpr int kRows = 4;

// 1 + exp(-t); the factors of t carry -log2(e), so that exp is one ex2.
template <int ACT>
__device__ __forceinline__ float act_denominator(float x) {
  constexpr float kLog2e = 1.4426950408889634f, kC1 = 2.f * 0.7978845608028654f, kC3 = kC1 * 0.044715f;
  const float t = ACT == SVDQ_ACT_SILU ? x * -kLog2e : x * fmaf(x * x, -kC3 * kLog2e, -kC1 * kLog2e);
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return 1.f + e;
}
__device__ __forceinline__ float rcp_approx_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <int ACT, bool GATED, bool LAM>
__global__ void __launch_bounds__(kThreads) glu_quant_kernel(GluParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int t = static_cast<int>(threadIdx.x);
  const int nc = p.K >> 3;
  const int cblocks = (nc + kThreads - 1) / kThreads;
  const int rb = static_cast<int>(blockIdx.x / static_cast<unsigned>(cblocks));
  const int c = static_cast<int>(blockIdx.x % static_cast<unsigned>(cblocks)) * kThreads + t;
  const int row0 = rb * kRows;
  if (row0 >= p.M) {      // the CTA behind the last row block
    fp8_zero_padding(p.scales, p.M, p.K, p.sfb, t, kThreads);
    return;
  }
  const bool on = c < nc;
  const size_t nscale = static_cast<size_t>((p.M + 127) / 128 * 128) * 4 * p.sfb;
  uint4 g[kRows], u[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = row0 + i;
    g[i] = on && row < p.M ? ld_global_v4_na(p.gate + static_cast<size_t>(row) * p.ldg + static_cast<size_t>(c) * 8)
                           : make_uint4(0, 0, 0, 0);
    if (GATED)
      u[i] = on && row < p.M ? ld_global_v4_na(p.up + static_cast<size_t>(row) * p.ldu + static_cast<size_t>(c) * 8)
                             : make_uint4(0, 0, 0, 0);
  }
  float lam[8];
  if (LAM) {
    const float4 l0 = on ? __ldg(reinterpret_cast<const float4*>(p.lam) + 2 * c) : make_float4(1.f, 1.f, 1.f, 1.f);
    const float4 l1 = on ? __ldg(reinterpret_cast<const float4*>(p.lam) + 2 * c + 1) : make_float4(1.f, 1.f, 1.f, 1.f);
    // reciprocals, used for kRows rows
    lam[0] = __frcp_rn(l0.x); lam[1] = __frcp_rn(l0.y); lam[2] = __frcp_rn(l0.z); lam[3] = __frcp_rn(l0.w);
    lam[4] = __frcp_rn(l1.x); lam[5] = __frcp_rn(l1.y); lam[6] = __frcp_rn(l1.z); lam[7] = __frcp_rn(l1.w);
  }
  const int G = p.K >> 7, pad = 4 * p.sfb - G;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = row0 + i;
    if (row >= p.M) break;                         // the same for every thread
    const uint32_t gx[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
    uint32_t ux[4] = {0, 0, 0, 0};
    if (GATED) { ux[0] = u[i].x; ux[1] = u[i].y; ux[2] = u[i].z; ux[3] = u[i].w; }
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = e & 1 ? bf16x2_hi(gx[e >> 1]) : bf16x2_lo(gx[e >> 1]);
      y[e] = x * rcp_approx_ftz(act_denominator<ACT>(x));
      if (GATED) y[e] *= e & 1 ? bf16x2_hi(ux[e >> 1]) : bf16x2_lo(ux[e >> 1]);
      if (LAM) y[e] *= lam[e];
    }
    fp8_store_chunk(y, on, row, c, p.K, p.sfb, p.codes, p.scales, nscale, p.err);
    if (c < pad) p.scales[fp8_sf_offset(row, G + c, p.sfb)] = 0;      // padding groups (c < 3)
  }
}

template <int ACT>
cudaError_t launch(const GluParams& p, const cudaLaunchConfig_t& cfg) {
  if (p.up) return p.lam ? cudaLaunchKernelEx(&cfg, glu_quant_kernel<ACT, true, true>, p)
                         : cudaLaunchKernelEx(&cfg, glu_quant_kernel<ACT, true, false>, p);
  return p.lam ? cudaLaunchKernelEx(&cfg, glu_quant_kernel<ACT, false, true>, p)
               : cudaLaunchKernelEx(&cfg, glu_quant_kernel<ACT, false, false>, p);
}

}  // namespace

cudaError_t launch_glu_quant(const GluParams& p, cudaStream_t s) {
  const int64_t cblocks = (p.K / 8 + kThreads - 1) / kThreads;
  const int64_t grid = cblocks * ((p.M + kRows - 1) / kRows) + (p.M % 128 ? 1 : 0);
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
  cudaError_t e = p.act == SVDQ_ACT_SILU ? launch<SVDQ_ACT_SILU>(p, cfg) : launch<SVDQ_ACT_GELU_TANH>(p, cfg);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace svdq
