// RMS norm with the residual's addition and an FP8 output (svdq_rmsnorm_quantize_act).
//
//   h = bf16(x + r),   y_k = (h_k * rsqrt(sum_k h_k^2 / K + eps)) * gamma_k,
//   codes = e4m3(y / 2^e), 2^e per 128 elements (fp8_quant.cuh).
//
// What bounds it: memory.  x and r are read once, h and the codes are written once: 7 bytes per
// element with a residual, 3 without.  One CTA holds one row in registers as bf16, adds the squares
// over the CTA, and quantizes from the registers: no second read.  Eight lanes hold a group of 128,
// two 16-byte chunks each, 64 elements apart so that the lanes of a load are neighbours; products run
// on pairs (f32x2).  Sixteen lanes to a group, with one chunk each and scalar products, take 56.9 us for
// 16384 x 3072 with residual against 54.9, and 80.2 us for 4608 x 12288 (rows x K here and below) against
// 64.3: twice as many lanes do shuffles and scale bytes.  Without a residual 4608 x 12288 takes 37 us where
// its bytes take 26: nothing is loaded while a CTA sums and quantizes its row.  Forming h gamma and the maxima before
// the CTA's sum is known saves work behind the barrier but keeps twice the registers: 60.2 and 66.5 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "fp8_quant.cuh"
#include "ptx.cuh"
#include "svdq_device.cuh"

namespace svdq {
namespace {

constexpr int kMaxThreads = 1024;

// bf16(a + b) of 8 elements
__device__ __forceinline__ uint4 add_bf16x8(uint4 a, uint4 b) {
  uint32_t x[4] = {a.x, a.y, a.z, a.w};
  const uint32_t y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __fadd2_rn(make_float2(bf16x2_lo(x[i]), bf16x2_hi(x[i])), make_float2(bf16x2_lo(y[i]), bf16x2_hi(y[i])));
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    x[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}
// Sum of the squares of 16 elements.
__device__ __forceinline__ float sumsq16(const uint4 (&h)[2]) {
  const uint32_t x[8] = {h[0].x, h[0].y, h[0].z, h[0].w, h[1].x, h[1].y, h[1].z, h[1].w};
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = make_float2(bf16x2_lo(x[i]), bf16x2_hi(x[i]));
    s = __ffma2_rn(f, f, s);
  }
  return s.x + s.y;
}
// y = (h rstd) gamma of 8 elements (gamma NULL: 1); returns max|y|.
__device__ __forceinline__ float normed8(uint4 h, float rstd, const float* gamma, float2 (&y)[4]) {
  const uint32_t x[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    y[i] = __fmul2_rn(make_float2(bf16x2_lo(x[i]), bf16x2_hi(x[i])), make_float2(rstd, rstd));
  if (gamma) {       // through the read-only path: every row reads it
    const float4 g0 = __ldg(reinterpret_cast<const float4*>(gamma)), g1 = __ldg(reinterpret_cast<const float4*>(gamma) + 1);
    y[0] = __fmul2_rn(y[0], make_float2(g0.x, g0.y));
    y[1] = __fmul2_rn(y[1], make_float2(g0.z, g0.w));
    y[2] = __fmul2_rn(y[2], make_float2(g1.x, g1.y));
    y[3] = __fmul2_rn(y[3], make_float2(g1.z, g1.w));
  }
  return fmaxf(fmaxf(fmaxf(fabsf(y[0].x), fabsf(y[0].y)), fmaxf(fabsf(y[1].x), fabsf(y[1].y))),
               fmaxf(fmaxf(fabsf(y[2].x), fabsf(y[2].y)), fmaxf(fabsf(y[3].x), fabsf(y[3].y))));
}
// Maximum over the 8 lanes that hold one group.
__device__ __forceinline__ float group_max8(float a) {
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
  return fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 4));
}
// Sum over the CTA of V values per thread, the same in every thread.  A value's place in the tree is that of
// its unit t + i * blockDim.x, whatever the number of threads: a row's sum does not depend on which launch
// shape takes it.
template <int V>
__device__ __forceinline__ float cta_sum(float (&s)[V]) {
  __shared__ float part[32 * V];
  const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
    if (lane == 0) part[(threadIdx.x >> 5) + i * nw] = s[i];
  }
  __syncthreads();
  float a = lane < nw * V ? part[lane] : 0.f;
  if (V > 1) a += lane + 32 < nw * V ? part[lane + 32] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  return a;
}

// VPT > 0: the row in registers; thread t has units t + i * blockDim.x, a unit being 16 elements of a
// group (8 at its column and 8 at 64 further).  VPT == 0: rows wider than the registers of a CTA; a
// second pass reads h again (from H where it was written, since H may have replaced an input).
// Registers: a CTA of 1024 threads may have 64 a thread; 40 and 52 let more CTAs share an SM (4608 x 3072
// takes 17.8 us with 40, 18.2 with 34 and 18.8 with 32; 4608 x 12288 64.6 us with 52, 76 with 58, 66 with 48).
template <int VPT>
__global__ void __maxnreg__(VPT == 2 ? 52 : 40) rmsnorm_quant_kernel(NormParams p) {
  constexpr int V = VPT > 0 ? VPT : 1;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int row = static_cast<int>(blockIdx.x);
  const int T = static_cast<int>(blockDim.x), t = static_cast<int>(threadIdx.x);
  if (row == p.M) {       // the CTA behind the last row
    fp8_zero_padding(p.scales, p.M, p.K, p.sfb, t, T);
    return;
  }
  const int G = p.K >> 7, units = G * 8;
  const __nv_bfloat16* x = p.X + static_cast<size_t>(row) * p.ldx;
  const __nv_bfloat16* r = p.R ? p.R + static_cast<size_t>(row) * p.ldr : nullptr;
  __nv_bfloat16* hout = p.H ? p.H + static_cast<size_t>(row) * p.ldh : nullptr;
  uint8_t* codes = p.codes + static_cast<size_t>(row) * p.K;
  // padding groups of this row
  if (t < 4 * p.sfb - G) p.scales[fp8_sf_offset(row, G + t, p.sfb)] = 0;
  auto column = [](int u) { return (u >> 3) * 128 + (u & 7) * 8; };
  // h of one unit of the row, from the inputs
  auto load = [&](int u, uint4 (&h)[2]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) h[q] = u < units ? ld_global_v4_na(x + column(u) + 64 * q) : make_uint4(0, 0, 0, 0);
  };
  auto add = [&](int u, uint4 (&h)[2], const uint4 (&rr)[2]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      h[q] = add_bf16x8(h[q], rr[q]);
      if (hout && u < units) *reinterpret_cast<uint4*>(hout + column(u) + 64 * q) = h[q];
    }
  };
  auto load_residual = [&](int u, uint4 (&rr)[2]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) rr[q] = u < units ? ld_global_v4_na(r + column(u) + 64 * q) : make_uint4(0, 0, 0, 0);
  };
  // norm, codes and scale of one unit; all lanes of the warp call it
  auto quantize = [&](int u, const uint4 (&h)[2], float rstd) {
    const bool on = u < units;
    const float* g = on && p.gamma ? p.gamma + column(u) : nullptr;
    float2 y[2][4];
    float a = normed8(h[0], rstd, g, y[0]);
    a = group_max8(fmaxf(a, normed8(h[1], rstd, g ? g + 64 : nullptr, y[1])));
    const uint32_t b = fp8_scale_byte(a);
    const float inv = fp8_inv_scale(b);
    if (on && SVDQ_IN_GLOBAL(column(u) + 72 <= p.K, p.err)) {
#pragma unroll
      for (int q = 0; q < 2; ++q) *reinterpret_cast<uint2*>(codes + column(u) + 64 * q) = fp8_codes8(y[q], inv);
      if ((u & 7) == 0) p.scales[fp8_sf_offset(row, u >> 3, p.sfb)] = static_cast<uint8_t>(b);
    }
  };
  float s[V];
  uint4 h[V][2];
  if (VPT > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) load(t + i * T, h[i]);
    if (r) {
      uint4 rr[V][2];
#pragma unroll
      for (int i = 0; i < V; ++i) load_residual(t + i * T, rr[i]);
#pragma unroll
      for (int i = 0; i < V; ++i) add(t + i * T, h[i], rr[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = sumsq16(h[i]);
  } else {
    s[0] = 0.f;
    for (int u = t; u < units; u += T) {
      load(u, h[0]);
      if (r) {
        uint4 rr[2];
        load_residual(u, rr);
        add(u, h[0], rr);
      }
      s[0] += sumsq16(h[0]);
    }
  }
  const float rstd = __frsqrt_rn(cta_sum(s) / static_cast<float>(p.K) + p.eps);
  if (VPT > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) quantize(t + i * T, h[i], rstd);
  } else {
    for (int u0 = 0; u0 < units; u0 += T) {
      const int u = u0 + t;
      if (hout) {
#pragma unroll
        for (int q = 0; q < 2; ++q) h[0][q] = u < units ? ld_global_v4_na(hout + column(u) + 64 * q) : make_uint4(0, 0, 0, 0);
      } else {
        load(u, h[0]);
        if (r) {
          uint4 rr[2];
          load_residual(u, rr);
          add(u, h[0], rr);
        }
      }
      quantize(u, h[0], rstd);
    }
  }
}

}  // namespace

cudaError_t launch_rmsnorm_quant(const NormParams& p, cudaStream_t s, int* variant) {
  // One unit per thread up to 256 threads, then two: with residual, 16384 x 3072 takes 54.9 us with 192
  // threads and 56.5 with 96, 8000 x 5120 47.7 us with 160 and 50.1 with 320, 4608 x 12288 64.3 us with 384
  // and 69.9 with 192 (four units).  Below 1024 rows, where a row's latency counts, one unit on up to 1024
  // threads (300 x 8192: 4.4 us against 5.6; 1000 x 8192: 11.5 against 13.2).
  const int units = p.K / 16;
  int vpt = units <= (p.M < 1024 ? kMaxThreads : 256) ? 1 : 2;
  if ((units + vpt - 1) / vpt > kMaxThreads) vpt = 0;
  *variant = vpt;
  const int threads = vpt > 0 ? ((units + vpt - 1) / vpt + 31) / 32 * 32 : kMaxThreads;
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
                             : cudaLaunchKernelEx(&cfg, rmsnorm_quant_kernel<2>, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace svdq
