// FP8 prologue: smoothing divide, quantization in groups of 128 and the low-rank down projection in
// one read of X (svdq_quantize_act_lowrank_down with SVDQ_FMT_FP8_G128).
//
//   X_hat = bf16(X / lambda),  codes = e4m3(X_hat / 2^e),  Z = bf16(X_hat L1^T).
//
// The data flow is that of "SVDQuant 阅读笔记" §6.1 "算法 2" steps 1-3.  Two kernels:
//
// With a branch.  A CTA owns 128 or 64 rows and, in a cluster of up to 8 CTAs that split K, a share of the
// 128-column groups.  TMA brings a group's X tile (two 128-byte-swizzled boxes of 64 columns) and
// L1 rows into a ring.  Sixteen warps, two sets in turn, form X_hat from shared memory: 16 neighbouring
// lanes hold one group of one row, so that a thread keeps its 8 columns' reciprocals over its rows, a
// row's codes leave as 128 contiguous bytes, and the group maximum takes four shuffles for two rows
// at once.  X_hat goes back to the place it came from, where the swizzle makes it the A operand of
// the tensor core: tcgen05 kind::f16 MMAs (M = 128, N = rank) accumulate Z in TMEM over the CTA's
// groups, so the branch costs the compute warps one 16-byte store per 8 elements.  The cluster's
// partial Z tiles are added by the CTA that owns the rows, in CTA order (deterministic).
//
// Without a branch.  Nothing is shared between threads but the group maximum: plain 16-byte loads,
// the same arithmetic, kQRows rows of the same 8 columns per thread.
//
// What bounds them.  Without a branch memory, 3 bytes per element: 16384 x 3072 takes 24.1 us (6.3 TB/s).
// The instructions around the codes decide how near it comes (8.6 per element; 11.8 took 29.5 us), so
// maxima are taken on bf16 pairs, two rows at a time, and one offset serves all of a thread's rows.
// With a branch the latency of a tile's way through the ring (TMA, shared memory to registers and back, MMA)
// with one CTA of 16 compute warps on an SM: 4608 x 3072 (rows x K), rank 32, takes 14.3 us, of which 2.4 pass
// before the first tile is there and 1.5 in the cluster's exchange; a tile of 64 rows takes 0.77 us, where
// its bytes would take 0.56, with issue slots 41% busy.  24 warps in three sets (15.4 us), eight lanes to a group (15.8) and more
// stages (14.6) give nothing there.
//
// The divide.  X_hat = bf16(RN_f32(x / lambda)) is formed as bf16(q), q = fma(x, yh, x yl), with
// yh = RD(1 / lambda) and yl = RN(yh (1 - lambda yh)) (the remainder is exact under FMA): yh + yl is
// 1 / lambda to 2^-45, so q's value before its rounding is within 2^-44 of the quotient, relatively.
// That gives the same bf16 always.  A difference would need the quotient that close to a point h where
// the two-step rounding changes, half an fp32 ulp beside a tie of bf16: h = (M 2^16 +- 1) 2^j with M
// odd, 257 <= M <= 511.  With the significands a of x (8 bits) and b of lambda (24 bits) as integers,
// b (M 2^16 +- 1) would have to lie within 2^5 of a multiple of 2^40.  Its low 16 bits are those of
// +-b, so b = B 2^16 + s with |s| <= 32 and B <= 256; then +-B + s M must vanish modulo 2^16, and
// |s| M <= 16352 leaves only s M = -+B, which M > B and B >= 128 rule out.  (The quotient
// must be a normal number well above 2^-126, like the remainder of any such divide.)  yl >= 0 keeps
// the sign of a zero.
#include <cuda.h>
#include <cuda_bf16.h>
#include <atomic>
#include <cstdint>

#include "fp8_quant.cuh"
#include "ptx.cuh"
#include "svdq_device.cuh"

namespace svdq {
namespace {

// ------------------------------------------------------------------ arithmetic shared by both kernels
// Reciprocals of a thread's 8 columns in two parts, as pairs.
struct Divisors {
  float2 yh[4], yl[4];
};
__device__ __forceinline__ float2 reciprocal2(float lam) {      // (yh, yl)
  const float yh = __frcp_rd(lam);
  return make_float2(yh, fmaf(-lam, yh, 1.f) * yh);
}
// X_hat of 8 elements: four bf16 pairs.
template <bool LAM>
__device__ __forceinline__ uint4 smooth8(uint4 v, const Divisors& d) {
  if (!LAM) return v;                                  // x / 1
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 a = make_float2(bf16x2_lo(w[e]), bf16x2_hi(w[e]));
    const float2 q = __ffma2_rn(a, d.yh[e], __fmul2_rn(a, d.yl[e]));
    const __nv_bfloat162 h = __floats2bfloat162_rn(q.x, q.y);
    w[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The pair of largest magnitude of either half, with signs that mean nothing (a NaN gives way to a number).
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_abs8(uint4 v) {
  return max_abs_bf16x2(max_abs_bf16x2(v.x, v.y), max_abs_bf16x2(v.z, v.w));
}
// Two rows' pairs a and b -> the bits of max|a| (low half) and max|b| (high half).  Bits of magnitudes
// order like the numbers, so that the group's maximum may be taken on them, two rows at a time.
__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) {
  return max_u16x2(__byte_perm(a, b, 0x5410) & 0x7FFF7FFFu, __byte_perm(a, b, 0x7632) & 0x7FFF7FFFu);
}
// The two rows' scale bytes, as 16-bit halves: fp8_scale_byte on the upper half of an fp32.
__device__ __forceinline__ uint32_t scale_bytes(uint32_t bits) {
  return max_u16x2(((bits + 0x001F001Fu) >> 7) & 0x01FF01FFu, 0x00080008u) - 0x00080008u;
}
__device__ __forceinline__ uint2 codes8(uint4 v, uint32_t byte) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float2 f[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = make_float2(bf16x2_lo(w[e]), bf16x2_hi(w[e]));
  return fp8_codes8(f, fp8_inv_scale(byte));
}

// ------------------------------------------------------------------ without a branch
constexpr int kQThreads = 128;
constexpr int kQRows = 4;

template <bool LAM>
__global__ void __launch_bounds__(kQThreads) quantize_fp8_kernel(const __nv_bfloat16* X, ProParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int t = static_cast<int>(threadIdx.x);
  const int nc = p.K >> 3, G = p.K >> 7, sfb = (p.K + 511) >> 9;
  const int cblocks = (nc + kQThreads - 1) / kQThreads;
  const int row0 = static_cast<int>(blockIdx.x / static_cast<unsigned>(cblocks)) * kQRows;
  const int c = static_cast<int>(blockIdx.x % static_cast<unsigned>(cblocks)) * kQThreads + t;
  uint8_t* scales = static_cast<uint8_t*>(p.scales);
  if (row0 >= p.M) {      // the CTA behind the last row block
    fp8_zero_padding(scales, p.M, p.K, sfb, t, kQThreads);
    return;
  }
  const bool on = c < nc;
  const int rows = min(kQRows, p.M - row0);
  uint4 v[kQRows];
#pragma unroll
  for (int i = 0; i < kQRows; ++i)
    v[i] = on && i < rows ? ld_global_v4_na(X + static_cast<size_t>(row0 + i) * p.K + static_cast<size_t>(c) * 8)
                          : make_uint4(0, 0, 0, 0);
  Divisors d;
  if (LAM) {
    const float4* lp = reinterpret_cast<const float4*>(p.lam) + (on ? 2 * c : 0);
    const float4 l0 = __ldg(lp), l1 = __ldg(lp + 1);
    const float l[8] = {l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 r0 = reciprocal2(l[2 * e]), r1 = reciprocal2(l[2 * e + 1]);
      d.yh[e] = make_float2(r0.x, r1.x);
      d.yl[e] = make_float2(r0.y, r1.y);
    }
  }
  uint32_t sb[kQRows / 2];
#pragma unroll
  for (int i = 0; i < kQRows; i += 2) {
    v[i] = smooth8<LAM>(v[i], d);
    v[i + 1] = smooth8<LAM>(v[i + 1], d);
    sb[i / 2] = max_bits(max_abs8(v[i]), max_abs8(v[i + 1]));
  }
#pragma unroll
  for (int o = 1; o <= 8; o <<= 1) {
#pragma unroll
    for (int i = 0; i < kQRows / 2; ++i) sb[i] = max_u16x2(sb[i], __shfl_xor_sync(0xffffffffu, sb[i], o));
  }
  if (!on) return;
#pragma unroll
  for (int i = 0; i < kQRows / 2; ++i) sb[i] = scale_bytes(sb[i]);
  uint8_t* dst = p.codes + static_cast<size_t>(row0) * p.K + static_cast<size_t>(c) * 8;
  // Lane 0 of a group has its byte; behind the row's last group the next lanes have the padding groups,
  // up to the next multiple of four, which is the same 4-byte word.
  const int grp = c >> 4, j = c & 15, nsc = grp == G - 1 ? 4 * sfb - grp : 1;
  uint8_t* sc = scales + fp8_sf_offset(row0, grp, sfb) + j;        // row0 is a multiple of 4: 16 bytes a row
#pragma unroll
  for (int i = 0; i < kQRows; ++i) {
    if (i >= rows) break;
    const uint32_t b = (sb[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
    if (SVDQ_IN_GLOBAL(c * 8 + 8 <= p.K, p.err)) *reinterpret_cast<uint2*>(dst) = codes8(v[i], b);
    dst += p.K;
    if (j < nsc) sc[16 * i] = j == 0 ? static_cast<uint8_t>(b) : 0;
  }
}

// ------------------------------------------------------------------ with a branch
constexpr int kComputeWarps = 16;
constexpr int kProdWarp = kComputeWarps, kMmaWarp = kComputeWarps + 1;
constexpr int kThreadsP = 32 * (kComputeWarps + 2);
constexpr int kMmaRows = 128;                           // rows of an MMA, see prologue_fp8_kernel
// An X tile of `rows` rows: two boxes of rows x 64 bf16.
__host__ __device__ constexpr uint32_t x_bytes(int rows) { return rows * 256u; }
constexpr uint32_t kLamBytes = 1024;                    // lambda and RN(1 / lambda) of 128 columns
constexpr int kMaxSplitP = 8;

__host__ __device__ constexpr uint32_t idesc_bf16p(int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}
// Padded row of a partial Z tile, in floats: 16 bytes more than the rank spread a column over the banks.
__host__ __device__ constexpr int zrow(int rank) { return rank + 4; }
__host__ __device__ constexpr uint32_t pstage_bytes(int rows, int rank) {
  return x_bytes(rows) + 256u * rank + kLamBytes;
}
// Partial sums that ks - 1 other CTAs send: [sender][a CTA's share of the rows][zrow].
__host__ __device__ constexpr uint32_t red_bytes(int rows, int rank, int ks) {
  return static_cast<uint32_t>((ks - 1) * ((rows + ks - 1) / ks) * zrow(rank) * 4);
}
__host__ __device__ constexpr uint32_t ptmem_cols(int rank) { return rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }
constexpr int kMaxStagesP = 6;            // even: a set of compute warps meets only its own slots, each in turn

struct PTail {
  uint64_t full[kMaxStagesP];     // X and L1 tiles (TMA) and the divisors (the producer's lanes) are there
  uint64_t xh_full[kMaxStagesP];  // X_hat has taken the place of X
  uint64_t empty[kMaxStagesP];    // the MMAs that read the stage have completed
  uint64_t acc_full;
  uint64_t red_full;              // the other CTAs' partial Z of this CTA's rows have arrived
  uint32_t tmem_base;
  int abort_flag;
};

// R rows per CTA, 128 or 64.  The MMAs have 128 rows either way: with R = 64 the upper half of the A
// tile is whatever follows in shared memory (the next box, L1, the next stage; slack behind the last)
// and the accumulator's upper lanes are not read.
template <bool LAM, int R>
__global__ void __launch_bounds__(kThreadsP, 1)
    prologue_fp8_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_l1,
                        ProParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int rank = p.rank, S = p.stages, ks = p.ksplit;
  constexpr uint32_t kXBytes = x_bytes(R);
  const uint32_t stage = pstage_bytes(R, rank);
  float* red = reinterpret_cast<float*>(smem + S * stage);
  PTail* sh = reinterpret_cast<PTail*>(smem + S * stage + red_bytes(R, rank, ks));
  volatile int* abort_flag = &sh->abort_flag;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int split = static_cast<int>(blockIdx.x) % ks;
  const int m0 = static_cast<int>(blockIdx.x) / ks * R;
  const int G = p.K >> 7, sfb = (p.K + 511) >> 9;
  const int gb = static_cast<int>(static_cast<int64_t>(G) * split / ks);                 // this CTA's groups
  const int ng = static_cast<int>(static_cast<int64_t>(G) * (split + 1) / ks) - gb;      // >= 1: ks <= G
  const int nrow = min(R, p.M - m0);
  // K split: CTA r adds up the Z rows [r share, r share + own) of the block
  const int share = (nrow + ks - 1) / ks;
  const int own = max(0, min(share, nrow - split * share));

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(&sh->full[s], 32);
      ptx::mbar_init(&sh->xh_full[s], kComputeWarps / 2);
      ptx::mbar_init(&sh->empty[s], 1);
    }
    ptx::mbar_init(&sh->acc_full, 1);
    ptx::mbar_init(&sh->red_full, 1);
    sh->abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&sh->tmem_base, ptmem_cols(rank));
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (ks > 1) {
    if (threadIdx.x == 0)
      ptx::mbar_arrive_expect_tx(&sh->red_full, static_cast<uint32_t>((ks - 1) * own * zrow(rank) * 4));
    ptx::cluster_arrive();                // waited for before anything is sent: every CTA has started
  }
  const uint32_t tmem = sh->tmem_base;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();

  if (warp == kProdWarp) {
    // ------------------------------------------------------------ producer: tiles and divisors
    if (lane == 0) {
      ptx::prefetch_tmap(&tmap_x);
      ptx::prefetch_tmap(&tmap_l1);
    }
    int s = 0;
    uint32_t ph = 1;
    // the next group's lambda is loaded while this one's tiles are on their way
    float l[4] = {1.f, 1.f, 1.f, 1.f};
    if (LAM)
#pragma unroll
      for (int i = 0; i < 4; ++i) l[i] = __ldg(p.lam + gb * 128 + i * 32 + lane);
    for (int g = 0; g < ng; ++g) {
      if (!wait_bounded_warp(&sh->empty[s], ph, abort_flag, p.err, kErrSiteProEmpty)) break;
      uint8_t* st = smem + s * stage;
      if (lane == 0) {
        ptx::mbar_expect_tx(&sh->full[s], kXBytes + 256u * rank);
        ptx::tma_load_3d(st, &tmap_x, &sh->full[s], 0, m0, 2 * (gb + g));
        ptx::tma_load_3d(st + kXBytes, &tmap_l1, &sh->full[s], 0, 0, 2 * (gb + g));
      }
      if (LAM) {
        float* ls = reinterpret_cast<float*>(st + kXBytes + 256 * rank);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (SVDQ_IN_SMEM(smem_raw, ls + 128 + i * 32 + lane, 4, p.err)) {
            const float2 y = reciprocal2(l[i]);
            ls[i * 32 + lane] = y.x;
            ls[128 + i * 32 + lane] = y.y;
          }
        }
        if (g + 1 < ng)
#pragma unroll
          for (int i = 0; i < 4; ++i) l[i] = __ldg(p.lam + (gb + g + 1) * 128 + i * 32 + lane);
      }
      ptx::mbar_arrive(&sh->full[s]);        // each lane releases its own stores
      if (++s == S) { s = 0; ph ^= 1u; }
    }
    end_issuing_role(abort_flag);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ Z += X_hat L1^T
    int s = 0;
    uint32_t ph = 0;
    const uint32_t idesc = idesc_bf16p(kMmaRows, rank);
    const uint64_t desc0 = ptx::sdesc_sw128(ptx::smem_u32(smem));
    for (int g = 0; g < ng; ++g) {
      if (!wait_bounded_warp(&sh->xh_full[s], ph, abort_flag, p.err, kErrSiteProPair)) break;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        const uint64_t ad = desc0 + static_cast<uint64_t>(s) * (stage / 16);
        const uint64_t bd = ad + kXBytes / 16;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            ptx::umma_f16(tmem, ad + h * (kXBytes / 32) + 2 * q, bd + static_cast<uint64_t>(h) * (8 * rank) + 2 * q,
                          idesc, (g | h | q) != 0 ? 1u : 0u);
        ptx::tc_commit(&sh->empty[s]);
        if (g == ng - 1) ptx::tc_commit(&sh->acc_full);
      }
      __syncwarp();
      if (++s == S) { s = 0; ph ^= 1u; }
    }
    end_issuing_role(abort_flag);
  } else {
    // ------------------------------------------------------------ compute warps
    // Two sets of eight warps take the tiles in turn, so that one set's waits and stores overlap the
    // other's arithmetic; a warp has an eighth of its set's tile's rows.
    constexpr int kSet = kComputeWarps / 2;
    const int set = warp / kSet;
    const int c = lane & 15;                               // 16-byte chunk of the 128-column group
    const int r0 = (warp % kSet) * (R / kSet) + (lane >> 4);       // rows r0, r0 + 2, ...
    uint8_t* scales = static_cast<uint8_t*>(p.scales);
    int s = set % S;
    uint32_t ph = static_cast<uint32_t>(set / S) & 1u;
    for (int g = set; g < ng; g += 2) {
      if (!wait_bounded_warp(&sh->full[s], ph, abort_flag, p.err, kErrSiteProFull)) {
        leave_aborted(abort_flag);
        break;
      }
      uint8_t* st = smem + s * stage;
      Divisors d;
      if (LAM) {
        const float4* ls = reinterpret_cast<const float4*>(st + kXBytes + 256 * rank) + 2 * c;
        const float4 h0 = ls[0], h1 = ls[1], l0 = ls[32], l1 = ls[33];
        d.yh[0] = make_float2(h0.x, h0.y);
        d.yh[1] = make_float2(h0.z, h0.w);
        d.yh[2] = make_float2(h1.x, h1.y);
        d.yh[3] = make_float2(h1.z, h1.w);
        d.yl[0] = make_float2(l0.x, l0.y);
        d.yl[1] = make_float2(l0.z, l0.w);
        d.yl[2] = make_float2(l1.x, l1.y);
        d.yl[3] = make_float2(l1.z, l1.w);
      }
      const int grp = gb + g;
      constexpr int kR = R / (2 * kSet);                   // rows of a thread
      uint4 v[kR];
      uint8_t* at0 = st + (c >> 3) * (kXBytes / 2) + r0 * 128;
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        uint8_t* at = at0 + i * 256 + (((c & 7) ^ ((r0 + 2 * i) & 7)) << 4);
        v[i] = SVDQ_IN_SMEM(smem_raw, at, 16, p.err) ? *reinterpret_cast<const uint4*>(at) : make_uint4(0, 0, 0, 0);
      }
      uint32_t sb[kR / 2];
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        uint8_t* at = at0 + i * 256 + (((c & 7) ^ ((r0 + 2 * i) & 7)) << 4);
        v[i] = smooth8<LAM>(v[i], d);
        if (LAM && SVDQ_IN_SMEM(smem_raw, at, 16, p.err)) *reinterpret_cast<uint4*>(at) = v[i];
      }
#pragma unroll
      for (int i = 0; i < kR; i += 2) sb[i / 2] = max_bits(max_abs8(v[i]), max_abs8(v[i + 1]));
      // X_hat is in place: hand the stage to the MMA warp before the codes are formed
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh->xh_full[s]);
#pragma unroll
      for (int o = 1; o <= 8; o <<= 1) {
#pragma unroll
        for (int i = 0; i < kR / 2; ++i) sb[i] = max_u16x2(sb[i], __shfl_xor_sync(0xffffffffu, sb[i], o));
      }
#pragma unroll
      for (int i = 0; i < kR / 2; ++i) sb[i] = scale_bytes(sb[i]);
      uint8_t* dst = p.codes + static_cast<size_t>(m0 + r0) * p.K + grp * 128 + c * 8;
      // Lane 0 of a group has its byte, the next ones those of the padding groups behind the last group
      // (the same 4-byte word).  A warp's rows are in one run of 32: 16 bytes a row.  Rows past M read as
      // zeros and get byte 0.
      const int nsc = grp == G - 1 ? 4 * sfb - grp : 1;
      uint8_t* sc = scales + fp8_sf_offset(m0 + r0, grp, sfb) + c;
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const uint32_t b = (sb[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
        if (m0 + r0 + 2 * i < p.M && SVDQ_IN_GLOBAL(grp < G, p.err)) *reinterpret_cast<uint2*>(dst) = codes8(v[i], b);
        dst += 2 * static_cast<size_t>(p.K);
        if (c < nsc) sc[32 * i] = c == 0 ? static_cast<uint8_t>(b) : 0;
      }
      s += 2;                                              // S >= 2
      if (s >= S) { s -= S; ph ^= 1u; }
    }
    if (warp < 4) {
      // ---------------------------------------------------------- Z: thread = row, column = rank index
      if (ks > 1) ptx::cluster_wait();
      float* part = reinterpret_cast<float*>(smem);          // [row][zrow], in the drained ring
      if (wait_bounded_warp(&sh->acc_full, 0u, abort_flag, p.err, kErrSiteGemmAccFull)) {
        ptx::tc_fence_after();
        const int row = warp * 32 + lane;
        const uint32_t base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
#pragma unroll 1
        for (int q = 0; q < (row < R ? rank : 0); q += 16) {       // the same for a warp
          uint32_t z[16];
          ptx::tmem_ld_32x32b_x16(base + q, z);
          ptx::tmem_wait_ld();
          float4* dst = reinterpret_cast<float4*>(part + row * zrow(rank) + q);
          if (SVDQ_IN_SMEM(smem_raw, dst, 64, p.err))
#pragma unroll
            for (int e = 0; e < 4; ++e)
              dst[e] = make_float4(__uint_as_float(z[4 * e]), __uint_as_float(z[4 * e + 1]),
                                   __uint_as_float(z[4 * e + 2]), __uint_as_float(z[4 * e + 3]));
        }
        ptx::tc_fence_before();
      } else {
        leave_aborted(abort_flag);
      }
      if (ks > 1) {
        // every other CTA gets its rows with one bulk copy
        ptx::fence_proxy_async_smem();
        named_barrier_sync(1, 128);
        if (warp == 0 && lane < ks && lane != split && *abort_flag == 0) {
          const int rows = min(share, nrow - lane * share);
          if (rows > 0)
            ptx::bulk_copy_to_cta(
                ptx::mapa_shared(ptx::smem_u32(red + (split - (split > lane ? 1 : 0)) * share * zrow(rank)),
                                 static_cast<uint32_t>(lane)),
                part + lane * share * zrow(rank), static_cast<uint32_t>(rows * zrow(rank) * 4),
                ptx::mapa_shared(ptx::smem_u32(&sh->red_full), static_cast<uint32_t>(lane)));
        }
        __syncwarp();
      }
    }
  }

  if (ks > 1 && warp >= 4) ptx::cluster_wait();              // warps 0-3 have waited
  __syncthreads();
  bool ok = *abort_flag == 0;
  if (ks > 1) {
    if (!wait_bounded_warp(&sh->red_full, 0u, abort_flag, p.err, kErrSiteGemmAccFinal)) {
      ok = false;
      leave_aborted(abort_flag);
    }
    // what the others sent has arrived; when all CTAs say so, every copy has left its source
    __syncwarp();
    ptx::cluster_arrive();
  }
  if (ok) {
    const float* mine = reinterpret_cast<const float*>(smem) + split * share * zrow(rank);
    const int per = rank / 4;                                // threads of a row, four columns each
    for (int i = threadIdx.x; i < own * per; i += kThreadsP) {
      const int r = i / per, q = i % per * 4;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int x = 0; x < ks; ++x) {
        const float* src = (x == split ? mine : red + (x - (x > split ? 1 : 0)) * share * zrow(rank)) + r * zrow(rank) + q;
        if (!SVDQ_IN_SMEM(smem_raw, src, 16, p.err)) continue;
        const float4 v = *reinterpret_cast<const float4*>(src);
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
      const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y), hi = __floats2bfloat162_rn(a.z, a.w);
      *reinterpret_cast<uint2*>(p.Z + static_cast<size_t>(m0 + split * share + r) * rank + q) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
  }
  __syncwarp();
  if (ks > 1) ptx::cluster_wait();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, ptmem_cols(rank));
  }
}

size_t psmem(int rows, int rank, int stages, int ks) {
  // the slack lets the unused half of the last stage's A tile be read
  return 1024 + static_cast<size_t>(stages) * pstage_bytes(rows, rank) + red_bytes(rows, rank, ks) + sizeof(PTail) +
         (rows < kMmaRows ? x_bytes(kMmaRows) - x_bytes(rows) : 0);
}
constexpr size_t kSmemMax = 232448;
// Six stages where they fit next to the partial sums, else four or two: an even
// number.  4608 x 12288, rank 32 without lambda, is bound by the loads: 31.8 us with six, 34.1 with four.
// The ring also holds a CTA's own partial tile.
int pstages(int rows, int rank, int ks) {
  int s = kMaxStagesP;
  while (s > 2 && psmem(rows, rank, s, ks) > kSmemMax) s -= 2;
  return s;
}
static_assert(1024 + 2 * pstage_bytes(128, 128) + red_bytes(128, 128, kMaxSplitP) + sizeof(PTail) <= kSmemMax,
              "two stages always fit");
static_assert(128 * zrow(128) * 4 <= 2 * pstage_bytes(128, 128) && 64 * zrow(128) * 4 <= 2 * pstage_bytes(64, 128) &&
                  128 * zrow(16) * 4 <= 2 * pstage_bytes(128, 16) && 64 * zrow(16) * 4 <= 2 * pstage_bytes(64, 16),
              "a partial Z tile in the ring");

template <bool LAM, int R>
void fill_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], int blocks, int ks, size_t smem,
                 cudaStream_t s) {
  cfg.gridDim = dim3(static_cast<unsigned>(blocks) * static_cast<unsigned>(ks), 1, 1);
  cfg.blockDim = dim3(kThreadsP, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
}

// Clusters of ks CTAs that the current device holds at once (0 on error), asked once per device.
int resident_clusters(int ks) {
  static std::atomic<int> cache[64][kMaxSplitP + 1];     // 0: not asked yet, else 1 + the figure
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int known = cache[dev][ks].load(std::memory_order_relaxed);
  if (known > 0) return known - 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  fill_config<true, 128>(cfg, attr, 1, ks, kSmemMax, nullptr);
  cfg.numAttrs = 1;                                      // the cluster alone
  int n = 0;
  if (set_smem_limit_once(reinterpret_cast<const void*>(prologue_fp8_kernel<true, 128>), kSmemMax) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, prologue_fp8_kernel<true, 128>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  cache[dev][ks].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <bool LAM, int R>
cudaError_t launch_branch(const CUtensorMap& tx, const CUtensorMap& tl1, ProParams p, cudaStream_t s) {
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(prologue_fp8_kernel<LAM, R>), kSmemMax);
  if (e != cudaSuccess) return e;
  p.stages = pstages(R, p.rank, p.ksplit);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  fill_config<LAM, R>(cfg, attr, p.Mpad / R, p.ksplit, psmem(R, p.rank, p.stages, p.ksplit), s);
  e = cudaLaunchKernelEx(&cfg, prologue_fp8_kernel<LAM, R>, tx, tl1, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

int prologue_fp8_rows(int M, int K, int num_sms, int* ksplit) {
  // 128 or 64 rows per CTA and the widest K split with every cluster resident at once: the least time
  // by rows x groups of a CTA x waves (4608 x 3072, rank 32: 36 blocks of 128 rows split by 3 leave
  // 40 of 148 SMs idle, 72 of 64 rows split by 2 leave 4).
  const int G = K / 128;
  int64_t best = 0;
  int rows = 0;
  for (int r : {128, 64}) {
    const int64_t blocks = (static_cast<int64_t>(M) + 127) / 128 * (128 / r);
    int ks = 1;
    for (int k = G < kMaxSplitP ? G : kMaxSplitP; k > 1; --k)
      if (resident_clusters(k) >= blocks) {
        ks = k;
        break;
      }
    const int64_t waves = ks > 1 ? 1 : (blocks + num_sms - 1) / num_sms;
    const int64_t cost = waves * r * ((G + ks - 1) / ks);
    if (rows == 0 || cost < best) {
      best = cost;
      rows = r;
      *ksplit = ks;
    }
  }
  return rows;
}

cudaError_t launch_prologue_fp8(int rows, const CUtensorMap& tx, const CUtensorMap& tl1, const ProParams& p,
                                cudaStream_t s) {
  if (rows == 128) return p.lam ? launch_branch<true, 128>(tx, tl1, p, s) : launch_branch<false, 128>(tx, tl1, p, s);
  return p.lam ? launch_branch<true, 64>(tx, tl1, p, s) : launch_branch<false, 64>(tx, tl1, p, s);
}

cudaError_t launch_quantize_fp8(const void* X, const ProParams& p, cudaStream_t s) {
  const int64_t cblocks = (p.K / 8 + kQThreads - 1) / kQThreads;
  const int64_t grid = cblocks * ((p.M + kQRows - 1) / kQRows) + (p.M % 128 ? 1 : 0);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kQThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(X);
  cudaError_t e = p.lam ? cudaLaunchKernelEx(&cfg, quantize_fp8_kernel<true>, x, p)
                        : cudaLaunchKernelEx(&cfg, quantize_fp8_kernel<false>, x, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace svdq
