// Device helpers of the kernels that write FP8 activations: the E8M0 scale of a 128-element
// group, the E4M3 codes under it, and the byte layout of the scales.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "ptx.cuh"
#include "svdq_device.cuh"

namespace svdq {

// E8M0 byte e + 127 of the smallest e >= -127 with a <= 448 * 2^e, for a >= 0: with a = f 2^(E - 127),
// f in [1, 2), and 448 = 1.75 * 2^8, e + 127 is E - 8, one more when f > 1.75: adding a quarter less
// one unit to the mantissa carries just then.  Zero and subnormal a have E <= 1 there and get byte 0.
__device__ __forceinline__ uint32_t fp8_scale_byte(float a) {
  return max((__float_as_uint(a) + 0x1FFFFFu) >> 23, 8u) - 8u;
}
// 2^-e for the byte e + 127 (0..248): the exponent field 254 - byte is that of a normal number,
// so multiplying by it divides by the scale exactly.
__device__ __forceinline__ float fp8_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Byte offset of (row, group) in the blocked FP8 scale layout; sfb = ceil(K/512) blocks per 128 rows.
// Rows of one run of 32 (row >> 5 the same) are 16 bytes apart.
__device__ __forceinline__ size_t fp8_sf_offset(int row, int grp, int sfb) {
  return (static_cast<size_t>(row >> 7) * sfb + (grp >> 2)) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4 +
         (grp & 3);
}

__device__ __forceinline__ float bf16x2_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16x2_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// 16 bytes that are read once: no line is kept in L1.  A plain load, not the read-only path: the
// same thread may later write to the address (an output in place).
__device__ __forceinline__ uint4 ld_global_v4_na(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Larger of two unsigned 16-bit halves each, one instruction.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Codes v inv of 8 elements.
__device__ __forceinline__ uint2 fp8_codes8(const float2 (&v)[4], float inv) {
  const float2 s = make_float2(inv, inv);
  return make_uint2(ptx::cvt_e4m3x4(__fmul2_rn(v[0], s), __fmul2_rn(v[1], s)),
                    ptx::cvt_e4m3x4(__fmul2_rn(v[2], s), __fmul2_rn(v[3], s)));
}

// Zero scale bytes of the padding: thread t of n writes its share of the padding rows M .. Mpad-1
// (a 4-byte word per row and block of groups) and of the padding groups of the rows below M.
__device__ __forceinline__ void fp8_zero_padding(uint8_t* scales, int M, int K, int sfb, int64_t t, int64_t n) {
  const int Mpad = (M + 127) / 128 * 128;
  const int64_t words = static_cast<int64_t>(Mpad - M) * sfb;
  for (int64_t i = t; i < words; i += n)
    *reinterpret_cast<uint32_t*>(scales + fp8_sf_offset(M + static_cast<int>(i / sfb), 4 * static_cast<int>(i % sfb), sfb)) = 0u;
}

}  // namespace svdq
