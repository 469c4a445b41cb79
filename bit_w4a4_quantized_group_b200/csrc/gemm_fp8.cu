// FP8 GEMM with the fused low-rank up projection (sm_100a, CTA pairs).
//
//   Y = bf16( sum_G 2^(e_x + e_w) sum_{k in G} q_x q_w + Z L2^T + bias ),   G = 128 elements of K.
//
// The scales are powers of two stored as E8M0 bytes, the scale type of kind::mxf8f6f4, so the
// tensor cores apply them and one fp32 TMEM accumulator takes the whole of K: there is no
// per-group promotion in the epilogue.  That kind wants one scale per row and 32 elements of K;
// here the four MMAs (K = 32 each) of a 128-element group simply name the same byte, and a
// 4-byte scale column, as tcgen05.cp brings it from a 128-row x 4-group block, serves 512
// elements of K.
//
// Design:
//   * clusters of two CTAs compute 256 x BN output tiles, BN = 64, 128, 192, 256 or 384 (the last as
//     two MMAs of 192 columns that share A), with cta_group::2 MMAs, each CTA holding 128 rows of A
//     and BN/2 rows of B; persistent clusters take contiguous runs of the N-fastest tile numbering.
//     What bounds large products is power: at 1000 W the SM clock falls to 1.3 GHz, and the energy
//     of moving operands from L2 counts beside that of the MMAs.  A step moves 128 + BN/2 rows per
//     SM for 128 x BN outputs, so 384 columns save 17% of the bytes of 256: 155 -> 144 us at
//     4608 x 12288 x 3072 back to back, 475 -> 427 at 16384 x 3072 x 9216;
//   * a ring slot holds two K steps (384 columns: one) of 128 bytes per row of A and B, each operand
//     brought by one 3-D TMA load ([K/128 chunks][rows][128 bytes], two chunks per box) and counted
//     on a barrier of the leader CTA (each CTA loads into its own shared memory; no multicast
//     loads).  The MMA warp's own work per slot (waits, issue, commit) is of the order of 400 cycles, so that slots of one
//     step kept the tensor pipe waiting: 512 cycles of MMAs at BN = 256, 128 at BN = 64;
//   * the scale blocks (512 bytes per 128 rows and four steps) have a ring of their own: a copy
//     warp of the leader moves them into the TMEM buffer of the same number (two or three
//     tcgen05.cp per four steps) as they land, ahead of the MMA warp;
//   * ceil(r/64) further slots hold Z and L2 (bf16): kind::f16 MMAs add the branch onto the same
//     accumulator;
//   * eight epilogue warps per CTA drain TMEM into registers, hand the accumulator back, add the
//     bias and store bf16 Y while the next tile's MMAs run.  192 columns and fewer leave TMEM for
//     two accumulators, so that the next tile's MMAs do not wait for the drain either; 256 and 384
//     columns have one, whose drain the MMAs wait for.
// Sizes in comments are M x K x N.
#include <cuda.h>
#include <cuda_bf16.h>
#include <atomic>
#include <cstdint>

#include "ptx.cuh"
#include "svdq_device.cuh"

namespace svdq {
namespace {

constexpr int kBM = 256;                      // pair tile rows
constexpr int kRows = 128;                    // A rows per CTA
constexpr int kKTile = 128;                   // E4M3 elements (bytes) per row and pipeline step
constexpr int kProdWarp = 0, kMmaWarp = 1, kCopyWarp = 2, kEpiWarp0 = 4;   // epilogue warps start at a multiple of 4
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);      // 384: up to 168 registers per thread
constexpr uint32_t kABytes = kRows * 128;
constexpr uint32_t kSfBlk = 512;              // scales of 128 rows x 4 groups
constexpr int kSfBufs = 4;
constexpr uint32_t kTmemCols = 512;

template <int BN>
struct Cfg {
  static constexpr int kHalves = BN > 256 ? 2 : 1;                    // MMAs across the tile
  static constexpr int kN = BN / kHalves;                             // columns of an MMA
  static constexpr int kSteps = BN > 256 ? 1 : 2;                     // K steps per ring slot
  static constexpr int kBRows = kN / 2;                               // B rows per CTA and MMA
  static constexpr uint32_t kBHalfBytes = kBRows * 128;
  static constexpr uint32_t kBBytes = kHalves * kBHalfBytes;          // ... per step
  static constexpr int kSfbBlks = (BN + 127) / 128;                   // 128-row scale blocks a tile's columns touch
  static constexpr uint32_t kSfBytes = (1 + kSfbBlks) * kSfBlk;
  static constexpr uint32_t kSfBufCols = 4 + 4 * kSfbBlks;            // A-scales 4 columns, B-scales 4 per block
  static constexpr uint32_t kStageBytes = kSteps * (kABytes + kBBytes);   // [A steps][B half 0 steps][B half 1 steps]
  static constexpr int kStages = BN == 384 ? 5 : BN >= 192 ? 3 : BN == 128 ? 4 : 5;
  static constexpr int kAccs = BN >= 256 ? 1 : 2;                     // accumulators in TMEM
  static constexpr uint32_t kTmemSf0 = kAccs * BN;
  static constexpr int kColsPerWarp = BN / 2;                         // epilogue columns of a warp
  static_assert(kTmemSf0 + kSfBufs * kSfBufCols <= kTmemCols, "TMEM");
};

// E4M3 x E4M3 with UE8M0 scales (bit 23); sf_id (bits 29-30 for A, 4-5 for B) selects the byte of
// the TMEM scale columns.
__host__ __device__ constexpr uint32_t idesc_mxf8(int m, int n, uint32_t sf_id) {
  return (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(m >> 4) << 24) | (sf_id << 29) |
         (sf_id << 4);
}
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n) {
  // bf16 x bf16 -> fp32, K-major A and B
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

template <int BN>
struct SharedTail {
  uint64_t full[Cfg<BN>::kStages];    // slot holds its two steps (TMA bytes of both CTAs)
  uint64_t empty[Cfg<BN>::kStages];   // the MMAs that read the slot have completed
  uint64_t sf_full[kSfBufs];          // scale slot holds the blocks of four steps (TMA bytes of both CTAs)
  uint64_t sf_ready[kSfBufs];         // ... and so does the TMEM buffer of the same number
  uint64_t sf_free[kSfBufs];          // the MMAs that read the TMEM buffer have completed
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint32_t tmem_base;
  int abort_flag;
};

template <int BN>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                    const __grid_constant__ CUtensorMap tmap_sfa, const __grid_constant__ CUtensorMap tmap_sfb,
                    const __grid_constant__ CUtensorMap tmap_z, const __grid_constant__ CUtensorMap tmap_l2,
                    GemmParams p) {
  using C = Cfg<BN>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sf_smem = smem + C::kStages * C::kStageBytes;
  SharedTail<BN>* sh = reinterpret_cast<SharedTail<BN>*>(sf_smem + kSfBufs * C::kSfBytes);
  volatile int* abort_flag = &sh->abort_flag;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();      // 0 = leader of the pair
  const int cluster = blockIdx.x >> 1;
  const int nclusters = gridDim.x >> 1;
  const int nk = p.K / kKTile;
  const int nd = (nk + C::kSteps - 1) / C::kSteps;   // slots of the 8-bit product per tile
  const int nk_lr = (p.rank + 63) / 64;              // ... and one per 64 columns of the branch
  constexpr int kSfSlots = 4 / C::kSteps;            // slots that a scale block serves
  const TileSeq tiles(p.num_tiles, p.tiles_n, cluster, nclusters);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&sh->full[s], 1);
      ptx::mbar_init(&sh->empty[s], 1);
    }
    for (int b = 0; b < kSfBufs; ++b) {
      ptx::mbar_init(&sh->sf_full[b], 1);
      ptx::mbar_init(&sh->sf_ready[b], 1);
      ptx::mbar_init(&sh->sf_free[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&sh->acc_full[b], 1);
      ptx::mbar_init(&sh->acc_empty[b], 2 * kEpiWarps);
    }
    sh->abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc_pair(&sh->tmem_base, kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  // the next kernel may set itself up on SMs that this grid leaves free; the set-up above may itself
  // have overlapped the end of the kernel that writes A and Z
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();

  if (warp == kProdWarp) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (lane == 0) {
      ptx::prefetch_tmap(&tmap_a);
      ptx::prefetch_tmap(&tmap_b);
      ptx::prefetch_tmap(&tmap_sfa);
      ptx::prefetch_tmap(&tmap_sfb);
      if (nk_lr > 0) {
        ptx::prefetch_tmap(&tmap_z);
        ptx::prefetch_tmap(&tmap_l2);
      }
      const uint64_t keep = ptx::l2_evict_last_policy();   // A and B tiles are re-read by other clusters
      int s = 0, b = 0;
      uint32_t ph = 1, sfph = 1;
      bool ok = true;
      for (int j = 0; j < tiles.count && ok; ++j) {
        const int m0 = tiles.mb(j) * kBM + static_cast<int>(rank) * kRows;     // this CTA's A rows
        const int n0 = tiles.nb(j) * BN;
        const int nb0 = n0 + static_cast<int>(rank) * C::kBRows;               // this CTA's B rows (+ kN for half 1)
        for (int d = 0; d < nd + nk_lr; ++d) {
          if (!wait_bounded(&sh->empty[s], ph, abort_flag, p.err, kErrSiteGemmEmpty)) { ok = false; break; }
          if (d < nd && d % kSfSlots == 0) {
            // the scale blocks of the next four steps
            if (!wait_bounded(&sh->sf_free[b], sfph, abort_flag, p.err, kErrSiteGemmSfFree)) { ok = false; break; }
            const uint32_t sf_leader = ptx::mapa_shared(ptx::smem_u32(&sh->sf_full[b]), 0);
            const uint32_t sf = ptx::smem_u32(sf_smem + b * C::kSfBytes);
            if (rank == 0) ptx::mbar_arrive_expect_tx(&sh->sf_full[b], 2 * C::kSfBytes);
            ptx::tma_load_3d_pair_hint(sf, &tmap_sfa, sf_leader, 0, d / kSfSlots, m0 >> 7, keep);
            ptx::tma_load_3d_pair_hint(sf + kSfBlk, &tmap_sfb, sf_leader, 0, d / kSfSlots, n0 >> 7, keep);
            if (++b == kSfBufs) { b = 0; sfph ^= 1u; }
          }
          const uint32_t full_leader = ptx::mapa_shared(ptx::smem_u32(&sh->full[s]), 0);
          const uint32_t st = ptx::smem_u32(smem + s * C::kStageBytes);
          if (d < nd) {
            // one load per operand and half: all steps of the slot (a missing second step reads as zeros)
            if (rank == 0) ptx::mbar_arrive_expect_tx(&sh->full[s], 2 * C::kStageBytes);
            ptx::tma_load_3d_pair_hint(st, &tmap_a, full_leader, 0, m0, C::kSteps * d, keep);
#pragma unroll
            for (int hh = 0; hh < C::kHalves; ++hh)
              ptx::tma_load_3d_pair_hint(st + C::kSteps * (kABytes + hh * C::kBHalfBytes), &tmap_b, full_leader, 0,
                                         nb0 + hh * C::kN, C::kSteps * d, keep);
          } else {
            if (rank == 0) ptx::mbar_arrive_expect_tx(&sh->full[s], 2 * (kABytes + C::kBBytes));
            ptx::tma_load_2d_pair(st, &tmap_z, full_leader, (d - nd) * 64, m0);
#pragma unroll
            for (int hh = 0; hh < C::kHalves; ++hh)
              ptx::tma_load_2d_pair(st + C::kSteps * (kABytes + hh * C::kBHalfBytes), &tmap_l2, full_leader,
                                    (d - nd) * 64, nb0 + hh * C::kN);
          }
          if (++s == C::kStages) { s = 0; ph ^= 1u; }
        }
      }
    }
    __syncwarp();
    end_issuing_role(abort_flag);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer (leader CTA only)
    // The whole warp runs the loop and the waits; one elected thread issues.
    if (rank == 0) {
      int s = 0, b = 0;
      uint32_t ph = 0, sfph = 0;           // parities of the ring slot and of the scale buffer
      bool ok = true;
      const uint32_t id16 = idesc_bf16(kBM, C::kN);
      const uint64_t desc0 = ptx::sdesc_sw128(ptx::smem_u32(smem));   // + bytes / 16 for any slot
      for (int j = 0; j < tiles.count && ok; ++j) {
        const int a = C::kAccs == 2 ? (j & 1) : 0;
        const uint32_t use = static_cast<uint32_t>(C::kAccs == 2 ? j >> 1 : j);
        if (!wait_bounded_warp(&sh->acc_empty[a], (use & 1u) ^ 1u, abort_flag, p.err, kErrSiteGemmAccEmpty)) break;
        ptx::tc_fence_after();
        const uint32_t acc = tmem + static_cast<uint32_t>(a * BN);
        // a tile that starts inside a 128-row scale block (BN 64 and 192) skips the block's first columns
        const uint32_t sfb_skip = static_cast<uint32_t>((tiles.nb(j) * BN) & 127) / 32;
        for (int d = 0; d < nd + nk_lr; ++d) {
          if (!wait_bounded_warp(&sh->full[s], ph, abort_flag, p.err, kErrSiteGemmFull)) { ok = false; break; }
          const bool main_slot = d < nd;
          if (main_slot && d % kSfSlots == 0 &&
              !wait_bounded_warp(&sh->sf_ready[b], sfph, abort_flag, p.err, kErrSiteGemmSfReady)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const bool sf_done = main_slot && (d % kSfSlots == kSfSlots - 1 || d == nd - 1);
          if (ptx::elect_one()) {
            const uint64_t ad = desc0 + static_cast<uint64_t>(s) * (C::kStageBytes / 16);
            const uint64_t bd = ad + C::kSteps * kABytes / 16;
            if (main_slot) {
              const uint32_t sfa = tmem + C::kTmemSf0 + static_cast<uint32_t>(b) * C::kSfBufCols;
              const uint32_t sfb = sfa + 4 + sfb_skip;
              const uint32_t id0 = static_cast<uint32_t>(d % kSfSlots) * C::kSteps;    // byte of the scale columns
#pragma unroll
              for (int h = 0; h < C::kSteps; ++h) {
                if (h == 1 && 2 * d + 1 == nk) break;                   // an odd last step
                const uint32_t id = id0 + h;
                const uint32_t idesc = idesc_mxf8(kBM, C::kN, 0) | (id << 29) | (id << 4);
#pragma unroll
                for (int hh = 0; hh < C::kHalves; ++hh)
#pragma unroll
                  for (int q = 0; q < kKTile / 32; ++q)
                    ptx::umma_mxf8_pair(acc + hh * C::kN, ad + h * (kABytes / 16) + 2 * q,
                                        bd + (hh * C::kSteps + h) * (C::kBHalfBytes / 16) + 2 * q, idesc, sfa | (id << 30),
                                        (sfb + hh * (C::kN / 32)) | (id << 30), (d | h | q) != 0 ? 1u : 0u);
              }
              if (sf_done) ptx::tc_commit_pair(&sh->sf_free[b], 0x3);
            } else {
              const int nmma = min(64, p.rank - (d - nd) * 64) / 16;
#pragma unroll
              for (int hh = 0; hh < C::kHalves; ++hh)
                for (int q = 0; q < nmma; ++q)
                  ptx::umma_f16_pair(acc + hh * C::kN, ad + 2 * q, bd + hh * C::kSteps * (C::kBHalfBytes / 16) + 2 * q,
                                     id16, 1u);
            }
            ptx::tc_commit_pair(&sh->empty[s], 0x3);
            if (d == nd + nk_lr - 1) ptx::tc_commit_pair(&sh->acc_full[a], 0x3);
          }
          __syncwarp();
          if (sf_done && ++b == kSfBufs) { b = 0; sfph ^= 1u; }
          if (++s == C::kStages) { s = 0; ph ^= 1u; }
        }
      }
    }
    end_issuing_role(abort_flag);
  } else if (warp == kCopyWarp) {
    // ------------------------------------------------------------ scale copier (leader CTA only)
    // Scale slot b goes to TMEM buffer b in both CTAs.  The producers refill the slot only when the
    // MMAs that read the buffer have completed, so slot and buffer are free together.
    if (rank == 0) {
      int b = 0;
      uint32_t sfph = 0;
      const uint64_t sfdesc0 = ptx::sdesc_sf(ptx::smem_u32(sf_smem));
      const int blocks = tiles.count * ((nk + 3) / 4);
      for (int i = 0; i < blocks; ++i) {
        if (!wait_bounded_warp(&sh->sf_full[b], sfph, abort_flag, p.err, kErrSiteGemmFull)) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint64_t sd = sfdesc0 + static_cast<uint64_t>(b) * (C::kSfBytes / 16);
          const uint32_t sfa = tmem + C::kTmemSf0 + static_cast<uint32_t>(b) * C::kSfBufCols;
          ptx::tmem_cp_32x128b_warpx4_pair(sfa, sd);
#pragma unroll
          for (int q = 0; q < C::kSfbBlks; ++q)
            ptx::tmem_cp_32x128b_warpx4_pair(sfa + 4 + 4 * q, sd + kSfBlk / 16 * (1 + q));
          ptx::tc_commit_pair_local(&sh->sf_ready[b]);
        }
        __syncwarp();
        if (++b == kSfBufs) { b = 0; sfph ^= 1u; }
      }
    }
    end_issuing_role(abort_flag);
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------ epilogue (8 warps, both CTAs)
    const int q = warp & 3;                 // TMEM lane quarter this warp may access
    const int h = (warp - kEpiWarp0) >> 2;  // column half of the tile
    constexpr int NC = C::kColsPerWarp / 32;
    for (int j = 0; j < tiles.count; ++j) {
      const int a = C::kAccs == 2 ? (j & 1) : 0;
      const uint32_t use = static_cast<uint32_t>(C::kAccs == 2 ? j >> 1 : j);
      const int m0 = tiles.mb(j) * kBM + static_cast<int>(rank) * kRows;
      const int col0 = tiles.nb(j) * BN + h * C::kColsPerWarp;
      if (NC > 4 && p.bias && lane < 3 && col0 + lane * 64 < p.N) {
        // the bias is read before the release here: have its lines in L1 by then
        const unsigned short touch = __ldg(reinterpret_cast<const unsigned short*>(p.bias) + col0 + lane * 64);
        asm volatile("" ::"h"(touch));
      }
      if (!wait_bounded_warp(&sh->acc_full[a], use & 1u, abort_flag, p.err, kErrSiteGemmAccFull)) {
        leave_aborted(abort_flag);
        break;
      }
      ptx::tc_fence_after();
      const uint32_t base = tmem + (static_cast<uint32_t>(q * 32) << 16) + a * BN + h * C::kColsPerWarp;
      const int row = m0 + q * 32 + lane;
      __nv_bfloat16* yrow = p.Y + static_cast<size_t>(row) * p.N + col0;
      auto release = [&]() {       // the accumulator goes back to the MMA warp
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_peer(ptx::mapa_shared(ptx::smem_u32(&sh->acc_empty[a]), 0));
      };
      // 16 columns: + bias -> bf16 pairs
      auto convert = [&](const uint32_t* v, int cl, uint32_t* o) {
        float bv[16];
        if (p.bias && SVDQ_IN_GLOBAL(col0 + cl >= p.N || col0 + cl + 16 <= p.N, p.err) && col0 + cl < p.N) {
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            const uint4 braw = __ldg(reinterpret_cast<const uint4*>(p.bias + col0 + cl + 8 * hb));
            const uint32_t bw[4] = {braw.x, braw.y, braw.z, braw.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              bv[8 * hb + 2 * e] = __uint_as_float(bw[e] << 16);
              bv[8 * hb + 2 * e + 1] = __uint_as_float(bw[e] & 0xFFFF0000u);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) bv[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __nv_bfloat162 hv = __floats2bfloat162_rn(__uint_as_float(v[2 * e]) + bv[2 * e],
                                                          __uint_as_float(v[2 * e + 1]) + bv[2 * e + 1]);
          o[e] = *reinterpret_cast<const uint32_t*>(&hv);
        }
      };
      auto store = [&](const uint32_t (&o)[8], int cl) {
        if (row >= p.M || col0 + cl >= p.N) return;          // the last tiles may reach past M and N
        if (!SVDQ_IN_GLOBAL(col0 + cl + 16 <= p.N, p.err)) return;
        if (p.y_align32) {
          ptx::st_global_v8_na(yrow + cl, o);
        } else {
          *reinterpret_cast<uint4*>(yrow + cl) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(yrow + cl + 8) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      };
      if constexpr (NC <= 4) {
        // the warp's columns into registers as they are, converted after the release
        uint32_t v[NC][32];
#pragma unroll
        for (int c = 0; c < NC; ++c) ptx::tmem_ld_32x32b_x32(base + c * 32, v[c]);
        ptx::tmem_wait_ld();
        release();
#pragma unroll
        for (int c16 = 0; c16 < 2 * NC; ++c16) {
          uint32_t o[8];
          convert(&v[c16 / 2][c16 % 2 * 16], c16 * 16, o);
          store(o, c16 * 16);
        }
      } else {
        // 192 columns: as bf16 pairs, since the registers do not hold that many fp32 values; even so this
        // kernel spills 136 bytes a thread (168 registers), the narrower ones nothing
        uint32_t o[2 * NC][8];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          uint32_t v[32];
          ptx::tmem_ld_32x32b_x32(base + c * 32, v);
          ptx::tmem_wait_ld();
          convert(v, c * 32, o[2 * c]);
          convert(v + 16, c * 32 + 16, o[2 * c + 1]);
        }
        release();
#pragma unroll
        for (int c16 = 0; c16 < 2 * NC; ++c16) store(o[c16], c16 * 16);
      }
    }
  }

  // Both CTAs finished: every MMA has completed (each epilogue saw its last accumulator) and no
  // remote arrive is still in flight.
  ptx::tc_fence_before();
  ptx::cluster_sync();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

template <int BN>
size_t smem_bytes() {
  return 1024 + Cfg<BN>::kStages * Cfg<BN>::kStageBytes + kSfBufs * Cfg<BN>::kSfBytes + sizeof(SharedTail<BN>);
}

template <int BN>
int max_active_clusters(size_t smem) {
  static std::atomic<int> cache[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && cache[dev] > 0) return cache[dev];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, gemm_fp8_kernel<BN>, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 0;
  }
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

template <int BN>
cudaError_t launch(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tsfa, const CUtensorMap& tsfb,
                   const CUtensorMap& tz, const CUtensorMap& tl2, const GemmParams& p, int num_sms, cudaStream_t s) {
  const size_t smem = smem_bytes<BN>();
  static_assert(1024 + Cfg<BN>::kStages * Cfg<BN>::kStageBytes + kSfBufs * Cfg<BN>::kSfBytes + sizeof(SharedTail<BN>) <= 232448,
                "shared memory of one CTA");
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(gemm_fp8_kernel<BN>), smem);
  if (e != cudaSuccess) return e;
  int clusters = max_active_clusters<BN>(smem);
  if (clusters <= 0) clusters = num_sms / 2;
  if (clusters > p.num_tiles) clusters = p.num_tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // may start under the kernel before
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, gemm_fp8_kernel<BN>, ta, tb, tsfa, tsfb, tz, tl2, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

float gemm_fp8_tile(int M, int N, int K, int num_sms, int* bn) {
  // The tile width with the least time.  Waves of the persistent clusters times K steps times the time
  // of a step, 0.13 us + 1.53 ns per column, and 4 us to start and drain.  Measured back to back, us a
  // step for widths 384, 256, 192, 128 and 64: 0.75, 0.54, 0.43, 0.32 and 0.23 at 4608 x 12288 x 3072;
  // whole calls 7.8 us at 300 x 2176 x 1152 (64 wide), 12.0 at 256 x 3072 x 9216 (128), 12.9 at 1024 x
  // 3072 x 3072 (192), 22.9 at 2048 x 3072 x 3072 (384; 24.9 with 256).  The rule knows neither a tile's
  // drain nor the bytes of Y: both 4608-token products come out at 142 us (141 measured for K = 12288, 157
  // for N = 12288), and with a single K step it is far off (16384 x 128 x 12288: 24 us, 155 measured).
  const int64_t tm = (M + kBM - 1) / kBM;
  const int64_t slots = num_sms / 2 > 0 ? num_sms / 2 : 1;
  float best = 0.f;
  *bn = 0;
  for (int w : {384, 256, 192, 128, 64}) {
    const int64_t tiles = tm * ((N + w - 1) / w);
    const float t = 4.f + static_cast<float>((tiles + slots - 1) / slots * (K / kKTile)) * (0.13f + 0.00153f * w);
    if (*bn == 0 || t < best) {
      best = t;
      *bn = w;
    }
  }
  return best;
}

cudaError_t launch_gemm_fp8(int bn, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tsfa,
                            const CUtensorMap& tsfb, const CUtensorMap& tz, const CUtensorMap& tl2,
                            const GemmParams& p, int num_sms, cudaStream_t s) {
  switch (bn) {
    case 384: return launch<384>(ta, tb, tsfa, tsfb, tz, tl2, p, num_sms, s);
    case 256: return launch<256>(ta, tb, tsfa, tsfb, tz, tl2, p, num_sms, s);
    case 192: return launch<192>(ta, tb, tsfa, tsfb, tz, tl2, p, num_sms, s);
    case 128: return launch<128>(ta, tb, tsfa, tsfb, tz, tl2, p, num_sms, s);
    case 64: return launch<64>(ta, tb, tsfa, tsfb, tz, tl2, p, num_sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace svdq
