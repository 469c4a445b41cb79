// RMS norm with the residual's addition and an FP8 output (svdq_rmsnorm_quantize_act).
//
//   h = bf16(x + r),   y_k = (h_k * rsqrt(sum_k h_k^2 / K + eps)) * gamma_k,
//   codes = e4m3(y / 2^e), 2^e per 128 elements (fp8_quant.cuh).
//
// What bounds it: memory.  x and r are read once, h and the codes are written once: 7 bytes per
// element with a residual, 3 without, and a few dozen instructions.  One CTA holds one row in
// registers (8 elements per 16-byte load, as bf16 pairs, so that a row of 32768 elements fits
// 1024 threads), adds the squares over the CTA, and quantizes from the registers: no second
// read.  Sixteen neighbouring lanes hold a group of 128, so its maximum takes four shuffles.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "fp8_quant.cuh"
#include "ptx.cuh"
#include "svdq_device.cuh"

namespace svdq {
namespace {

constexpr int kMaxThreads = 1024;
// A thread keeps up to 8 chunks of 16 bytes in registers; with 8, of 256 threads at most.
constexpr int max_threads(int vpt) { return vpt == 8 ? 256 : kMaxThreads; }

__device__ __forceinline__ uint4 add_bf16x8(uint4 a, uint4 b) {
  uint32_t x[4] = {a.x, a.y, a.z, a.w};
  const uint32_t y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(bf16x2_lo(x[i]) + bf16x2_lo(y[i]), bf16x2_hi(x[i]) + bf16x2_hi(y[i]));
    x[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ float sumsq8(uint4 v, float s) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(bf16x2_lo(x[i]), bf16x2_lo(x[i]), s);
    s = fmaf(bf16x2_hi(x[i]), bf16x2_hi(x[i]), s);
  }
  return s;
}
// y = (h * rstd) * gamma of one chunk; gamma is read through the read-only path (every row reads it)
__device__ __forceinline__ void normed8(uint4 v, float rstd, const float* gamma, int c, float (&y)[8]) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = bf16x2_lo(x[i]) * rstd;
    y[2 * i + 1] = bf16x2_hi(x[i]) * rstd;
  }
  if (gamma) {
    const float4 g0 = __ldg(reinterpret_cast<const float4*>(gamma) + 2 * c);
    const float4 g1 = __ldg(reinterpret_cast<const float4*>(gamma) + 2 * c + 1);
    y[0] *= g0.x; y[1] *= g0.y; y[2] *= g0.z; y[3] *= g0.w;
    y[4] *= g1.x; y[5] *= g1.y; y[6] *= g1.z; y[7] *= g1.w;
  }
}
// Sum over the CTA, the same value in every thread; the order is fixed by the launch shape.
__device__ __forceinline__ float cta_sum(float s) {
  __shared__ float part[32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
  s = lane < nw ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// VPT > 0: the row in registers, chunk c = threadIdx.x + i * blockDim.x.  VPT == 0: rows wider than
// the registers of a CTA; a second pass reads h again (from H where it was written, since H may
// have replaced an input).
template <int VPT>
__global__ void __launch_bounds__(max_threads(VPT)) rmsnorm_quant_kernel(NormParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int row = static_cast<int>(blockIdx.x);
  const int T = static_cast<int>(blockDim.x), t = static_cast<int>(threadIdx.x);
  if (row == p.M) {       // the CTA behind the last row
    fp8_zero_padding(p.scales, p.M, p.K, p.sfb, t, T);
    return;
  }
  const int nc = p.K >> 3;
  const __nv_bfloat16* x = p.X + static_cast<size_t>(row) * p.ldx;
  const __nv_bfloat16* r = p.R ? p.R + static_cast<size_t>(row) * p.ldr : nullptr;
  __nv_bfloat16* hout = p.H ? p.H + static_cast<size_t>(row) * p.ldh : nullptr;
  const size_t nscale = static_cast<size_t>((p.M + 127) / 128 * 128) * 4 * p.sfb;
  // padding groups of this row
  if (t < 4 * p.sfb - (p.K >> 7)) p.scales[fp8_sf_offset(row, (p.K >> 7) + t, p.sfb)] = 0;
  float s = 0.f;
  uint4 h[VPT > 0 ? VPT : 1];
  if (VPT > 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * T;
      h[i] = c < nc ? ld_global_v4_na(x + static_cast<size_t>(c) * 8) : make_uint4(0, 0, 0, 0);
    }
    if (r) {
      uint4 rr[VPT > 0 ? VPT : 1];
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = t + i * T;
        rr[i] = c < nc ? ld_global_v4_na(r + static_cast<size_t>(c) * 8) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = t + i * T;
        h[i] = add_bf16x8(h[i], rr[i]);
        if (hout && c < nc) *reinterpret_cast<uint4*>(hout + static_cast<size_t>(c) * 8) = h[i];
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) s = sumsq8(h[i], s);
  } else {
    for (int c = t; c < nc; c += T) {
      uint4 v = ld_global_v4_na(x + static_cast<size_t>(c) * 8);
      if (r) {
        v = add_bf16x8(v, ld_global_v4_na(r + static_cast<size_t>(c) * 8));
        if (hout) *reinterpret_cast<uint4*>(hout + static_cast<size_t>(c) * 8) = v;
      }
      s = sumsq8(v, s);
    }
  }
  s = cta_sum(s);
  const float rstd = __frsqrt_rn(s / static_cast<float>(p.K) + p.eps);
  if (VPT > 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * T;
      const bool on = c < nc;
      float y[8];
      normed8(h[i], rstd, on ? p.gamma : nullptr, c, y);
      fp8_store_chunk(y, on, row, c, p.K, p.sfb, p.codes, p.scales, nscale, p.err);
    }
  } else {
    for (int c0 = 0; c0 < nc; c0 += T) {
      const int c = c0 + t;
      const bool on = c < nc;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (on) {
        if (hout) {
          v = ld_global_v4_na(hout + static_cast<size_t>(c) * 8);
        } else {
          v = ld_global_v4_na(x + static_cast<size_t>(c) * 8);
          if (r) v = add_bf16x8(v, ld_global_v4_na(r + static_cast<size_t>(c) * 8));
        }
      }
      float y[8];
      normed8(v, rstd, on ? p.gamma : nullptr, c, y);
      fp8_store_chunk(y, on, row, c, p.K, p.sfb, p.codes, p.scales, nscale, p.err);
    }
  }
}

}  // namespace

cudaError_t launch_rmsnorm_quant(const NormParams& p, cudaStream_t s) {
  // About 192 threads a row when there are rows for every SM several times over (16384 x 3072 with
  // residual: 56 us with 192 threads, 66 with 384; 4608 x 12288: see the header), one chunk per
  // thread, up to 1024, when a row's latency is all that counts (one row: 1.9 us against 2.2).
  const int nc = p.K / 8;
  const int want = p.M >= 1024 ? 192 : kMaxThreads;
  int vpt = 0, t = 0;
  for (int v : {1, 2, 3, 4, 8}) {
    const int need = (nc + v - 1) / v;
    if (need > max_threads(v)) continue;
    vpt = v;
    t = need;
    if (need <= want) break;
  }
  const int threads = vpt > 0 ? (t + 31) / 32 * 32 : kMaxThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.M) + (p.M % 128 ? 1u : 0u), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = vpt == 0   ? cudaLaunchKernelEx(&cfg, rmsnorm_quant_kernel<0>, p)
                  : vpt == 1 ? cudaLaunchKernelEx(&cfg, rmsnorm_quant_kernel<1>, p)
                  : vpt == 2 ? cudaLaunchKernelEx(&cfg, rmsnorm_quant_kernel<2>, p)
                  : vpt == 3 ? cudaLaunchKernelEx(&cfg, rmsnorm_quant_kernel<3>, p)
                  : vpt == 4 ? cudaLaunchKernelEx(&cfg, rmsnorm_quant_kernel<4>, p)
                             : cudaLaunchKernelEx(&cfg, rmsnorm_quant_kernel<8>, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace svdq
