// FP8 GEMM for few tokens (sm_100a): the same product as gemm_fp8.cu with the operands' roles
// exchanged.
//
// With few tokens the work is reading the weights once.  A 256-row tile of tokens would be nearly
// empty and leave too few tiles for the SMs, so here the weights are the 128-row operand of the MMA
// and the tokens its N side, T = 16, 32, 64 or 128 wide: D[n][m] = sum_k W[n][k] X[m][k].  The K
// steps of a tile are split over a cluster of up to 8 CTAs, so that about two CTAs per SM stream
// weights at once; with K = 4096 a CTA's whole share is in flight in its ring.  The CTAs' fp32
// partial tiles are added through distributed shared memory, in CTA order (deterministic), and
// the bias is added before the one rounding to bf16.
//
// Scales: as in gemm_fp8.cu a 512-byte block serves four K steps; a CTA whose share starts inside
// such a block loads that block with its first step.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"
#include "svdq_device.cuh"

namespace svdq {
namespace {

constexpr int kRowsW = 128;                   // weight rows per tile
constexpr int kKTile = 128;                   // E4M3 elements (bytes) per row and step
constexpr int kProdWarp = 0, kMmaWarp = 1, kCopyWarp = 2, kEpiWarp0 = 4;   // epilogue: 4 warps, one per lane quarter
constexpr int kThreads = 256;
constexpr uint32_t kWBytes = kRowsW * 128;
constexpr uint32_t kSfBlk = 512;
constexpr int kSfBufs = 4;

template <int T>
struct Cfg {
  static constexpr uint32_t kXBytes = T * 128;
  static constexpr uint32_t kStageBytes = kWBytes + kXBytes + 2 * kSfBlk;
  static constexpr int kStages = T <= 32 ? 5 : T == 64 ? 4 : 3;       // two CTAs per SM
  static constexpr uint32_t kTmemSf0 = T;
  static constexpr uint32_t kTmemCols = T <= 32 ? 64 : T == 64 ? 128 : 256;
  static_assert(T + kSfBufs * 8 <= kTmemCols, "TMEM");
  static_assert(T * kRowsW * 4 <= kStages * kStageBytes, "the partial tile reuses the ring");
};

__host__ __device__ constexpr uint32_t idesc_mxf8(int m, int n) {      // E4M3 x E4M3, UE8M0 scales
  return (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(m >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

template <int T>
struct SharedTail {
  uint64_t full[Cfg<T>::kStages];
  uint64_t empty[Cfg<T>::kStages];
  uint64_t sf_ready[kSfBufs];
  uint64_t sf_free[kSfBufs];
  uint64_t acc_full;
  uint32_t tmem_base;
  int abort_flag;
};

template <int T>
__global__ void __launch_bounds__(kThreads, 2)
    gemm_fp8_small_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                          const __grid_constant__ CUtensorMap tmap_sfw, const __grid_constant__ CUtensorMap tmap_sfx,
                          const __grid_constant__ CUtensorMap tmap_l2, const __grid_constant__ CUtensorMap tmap_z,
                          GemmParams p) {
  using C = Cfg<T>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  SharedTail<T>* sh = reinterpret_cast<SharedTail<T>*>(smem + C::kStages * C::kStageBytes);
  volatile int* abort_flag = &sh->abort_flag;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int ks = p.ksplit;
  const int split = static_cast<int>(blockIdx.x) % ks;        // rank in the cluster
  const int tile = static_cast<int>(blockIdx.x) / ks;
  const int n0 = (tile % p.tiles_n) * kRowsW;                 // neighbouring clusters share the tokens
  const int m0 = (tile / p.tiles_n) * T;
  const int nk_all = p.K / kKTile;
  const int kb = static_cast<int>(static_cast<int64_t>(nk_all) * split / ks);
  const int nk = static_cast<int>(static_cast<int64_t>(nk_all) * (split + 1) / ks) - kb;   // >= 1: ks <= nk_all
  const int nk_lr = split == ks - 1 ? (p.rank + 63) / 64 : 0; // the last CTA also takes the branch
  const int ntok = min(T, p.M - m0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&sh->full[s], 1);
      ptx::mbar_init(&sh->empty[s], 1);
    }
    for (int b = 0; b < kSfBufs; ++b) {
      ptx::mbar_init(&sh->sf_ready[b], 1);
      ptx::mbar_init(&sh->sf_free[b], 1);
    }
    ptx::mbar_init(&sh->acc_full, 1);
    sh->abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&sh->tmem_base, C::kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  ptx::griddep_launch_dependents();
  // the set-up above may overlap the end of the kernel that writes X and Z
  ptx::griddep_wait();

  // step k of this CTA (k < nk: the weights' K step kb + k) brings the scale blocks of the steps
  // up to the next multiple of four
  auto brings_scales = [&](int k) { return k < nk && (k == 0 || ((kb + k) & 3) == 0); };

  if (warp == kProdWarp) {
    if (lane == 0) {
      ptx::prefetch_tmap(&tmap_w);
      ptx::prefetch_tmap(&tmap_x);
      for (int k = 0; k < nk + nk_lr; ++k) {
        const int s = k % C::kStages;
        const uint32_t ph = (k / C::kStages) & 1;
        if (!wait_bounded(&sh->empty[s], ph ^ 1u, abort_flag, p.err, kErrSiteGemmEmpty)) break;
        uint8_t* st = smem + s * C::kStageBytes;
        const bool sf = brings_scales(k);
        ptx::mbar_arrive_expect_tx(&sh->full[s], kWBytes + C::kXBytes + (sf ? 2 * kSfBlk : 0u));
        if (k < nk) {
          ptx::tma_load_2d(st, &tmap_w, &sh->full[s], (kb + k) * kKTile, n0);
          ptx::tma_load_2d(st + kWBytes, &tmap_x, &sh->full[s], (kb + k) * kKTile, m0);
          if (sf) {
            ptx::tma_load_3d(st + kWBytes + C::kXBytes, &tmap_sfw, &sh->full[s], 0, (kb + k) >> 2, n0 >> 7);
            ptx::tma_load_3d(st + kWBytes + C::kXBytes + kSfBlk, &tmap_sfx, &sh->full[s], 0, (kb + k) >> 2, m0 >> 7);
          }
        } else {
          ptx::tma_load_2d(st, &tmap_l2, &sh->full[s], (k - nk) * 64, n0);
          ptx::tma_load_2d(st + kWBytes, &tmap_z, &sh->full[s], (k - nk) * 64, m0);
        }
      }
    }
    __syncwarp();
  } else if (warp == kCopyWarp) {
    int b = 0;
    uint32_t sfph = 1;
    const uint64_t sfdesc0 = ptx::sdesc_sf(ptx::smem_u32(smem) + kWBytes + C::kXBytes);
    for (int k = 0; k < nk; ++k) {
      if (!brings_scales(k)) continue;
      const int s = k % C::kStages;
      const uint32_t ph = (k / C::kStages) & 1;
      if (!wait_bounded(&sh->full[s], ph, abort_flag, p.err, kErrSiteGemmFull) ||
          !wait_bounded(&sh->sf_free[b], sfph, abort_flag, p.err, kErrSiteGemmSfFree))
        break;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        const uint64_t sd = sfdesc0 + static_cast<uint64_t>(s) * (C::kStageBytes / 16);
        const uint32_t sfa = tmem + C::kTmemSf0 + static_cast<uint32_t>(b) * 8;
        ptx::tmem_cp_32x128b_warpx4(sfa, sd);
        ptx::tmem_cp_32x128b_warpx4(sfa + 4, sd + kSfBlk / 16);
        ptx::tc_commit(&sh->sf_ready[b]);
      }
      __syncwarp();
      if (++b == kSfBufs) { b = 0; sfph ^= 1u; }
    }
  } else if (warp == kMmaWarp) {
    int s = 0, b = 0;
    uint32_t ph = 0, sfph = 0;
    const uint32_t id16 = idesc_bf16(kRowsW, T);
    const uint64_t desc0 = ptx::sdesc_sw128(ptx::smem_u32(smem));
    const uint32_t sfx_skip = static_cast<uint32_t>(m0 & 127) / 32;    // T = 16 has m0 = 0
    for (int k = 0; k < nk + nk_lr; ++k) {
      if (!wait_bounded(&sh->full[s], ph, abort_flag, p.err, kErrSiteGemmFull)) break;
      const bool main_step = k < nk;
      const uint32_t id = static_cast<uint32_t>((kb + k) & 3);
      if (brings_scales(k) && !wait_bounded(&sh->sf_ready[b], sfph, abort_flag, p.err, kErrSiteGemmSfReady)) break;
      ptx::tc_fence_after();
      const bool sf_done = main_step && (id == 3 || k == nk - 1);
      if (ptx::elect_one()) {
        const uint64_t wd = desc0 + static_cast<uint64_t>(s) * (C::kStageBytes / 16);
        const uint64_t xd = wd + kWBytes / 16;
        if (main_step) {
          const uint32_t sfa = tmem + C::kTmemSf0 + static_cast<uint32_t>(b) * 8;
          const uint32_t sfb = sfa + 4 + sfx_skip;
          const uint32_t idesc = idesc_mxf8(kRowsW, T) | (id << 29) | (id << 4);
#pragma unroll
          for (int q = 0; q < kKTile / 32; ++q)
            ptx::umma_mxf8(tmem, wd + 2 * q, xd + 2 * q, idesc, sfa | (id << 30), sfb | (id << 30),
                           (k | q) != 0 ? 1u : 0u);
          if (sf_done) ptx::tc_commit(&sh->sf_free[b]);
        } else {
          const int nmma = min(64, p.rank - (k - nk) * 64) / 16;
          for (int q = 0; q < nmma; ++q) ptx::umma_f16(tmem, wd + 2 * q, xd + 2 * q, id16, 1u);
        }
        ptx::tc_commit(&sh->empty[s]);
        if (k == nk + nk_lr - 1) ptx::tc_commit(&sh->acc_full);
      }
      __syncwarp();
      if (sf_done && ++b == kSfBufs) { b = 0; sfph ^= 1u; }
      if (++s == C::kStages) { s = 0; ph ^= 1u; }
    }
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------ thread = weight row, column = token
    const int q = warp & 3;
    const int n = q * 32 + lane;
    if (wait_bounded(&sh->acc_full, 0u, abort_flag, p.err, kErrSiteGemmAccFull)) {
      ptx::tc_fence_after();
      const uint32_t base = tmem + (static_cast<uint32_t>(q * 32) << 16);
      float* part = reinterpret_cast<float*>(smem);           // [token][128], the ring is drained
      const float bias = p.bias ? __bfloat162float(p.bias[n0 + n]) : 0.f;
#pragma unroll 1
      for (int c = 0; c < ntok; c += 16) {
        uint32_t v[16];
        ptx::tmem_ld_32x32b_x16(base + c, v);
        ptx::tmem_wait_ld();
        if (ks > 1) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (SVDQ_IN_SMEM(smem_raw, part + (c + e) * kRowsW + n, 4, p.err))
              part[(c + e) * kRowsW + n] = __uint_as_float(v[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (c + e < ntok && SVDQ_IN_GLOBAL(n0 + n < p.N, p.err))
              p.Y[static_cast<size_t>(m0 + c + e) * p.N + n0 + n] = __float2bfloat16_rn(__uint_as_float(v[e]) + bias);
        }
      }
      ptx::tc_fence_before();
    }
  }

  if (ks > 1) {
    // Partial tiles of the cluster's CTAs, added in CTA order: CTA r takes the tokens r, r + ks, ...
    // and a thread two neighbouring columns of one of them.
    ptx::cluster_sync();
    if (*abort_flag == 0) {
      const uint32_t part = ptx::smem_u32(smem);
      const int col = 2 * (threadIdx.x & 63);
      float b0 = 0.f, b1 = 0.f;
      if (p.bias) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p.bias + n0 + col));
        b0 = __uint_as_float(w << 16);
        b1 = __uint_as_float(w & 0xFFFF0000u);
      }
      for (int c = split + ks * (threadIdx.x >> 6); c < ntok; c += ks * (kThreads / 64)) {
        const uint32_t at = part + static_cast<uint32_t>(c * kRowsW + col) * 4;
        float2 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < ks) v[r] = ptx::ld_shared_cluster_v2f32(ptx::mapa_shared(at, static_cast<uint32_t>(r)));
        float s0 = v[0].x, s1 = v[0].y;
#pragma unroll
        for (int r = 1; r < 8; ++r)
          if (r < ks) {
            s0 += v[r].x;
            s1 += v[r].y;
          }
        if (SVDQ_IN_GLOBAL(n0 + col + 2 <= p.N, p.err))
          *reinterpret_cast<__nv_bfloat162*>(p.Y + static_cast<size_t>(m0 + c) * p.N + n0 + col) =
              __floats2bfloat162_rn(s0 + b0, s1 + b1);
      }
    }
    ptx::cluster_sync();                                       // peers keep their partials until read
  } else {
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int T>
cudaError_t launch(const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& tsfw, const CUtensorMap& tsfx,
                   const CUtensorMap& tl2, const CUtensorMap& tz, const GemmParams& p, cudaStream_t s) {
  constexpr size_t smem = 1024 + Cfg<T>::kStages * Cfg<T>::kStageBytes + sizeof(SharedTail<T>);
  static_assert(2 * (smem + 1024) <= 228 * 1024, "two CTAs per SM");
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(gemm_fp8_small_kernel<T>), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.num_tiles) * static_cast<unsigned>(p.ksplit), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.ksplit);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, gemm_fp8_small_kernel<T>, tw, tx, tsfw, tsfx, tl2, tz, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

int gemm_fp8_small_tokens(int M) {
  if (M > 128) return 0;
  return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
}

int gemm_fp8_small_split(int tiles, int K, int num_sms) {
  const int nk = K / kKTile;
  int ks = 2 * num_sms / tiles;
  if (ks > 8) ks = 8;
  if (ks > nk) ks = nk;
  return ks < 1 ? 1 : ks;
}

cudaError_t launch_gemm_fp8_small(int tokens, const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& tsfw,
                                  const CUtensorMap& tsfx, const CUtensorMap& tl2, const CUtensorMap& tz,
                                  const GemmParams& p, cudaStream_t s) {
  switch (tokens) {
    case 16: return launch<16>(tw, tx, tsfw, tsfx, tl2, tz, p, s);
    case 32: return launch<32>(tw, tx, tsfw, tsfx, tl2, tz, p, s);
    case 64: return launch<64>(tw, tx, tsfw, tsfx, tl2, tz, p, s);
    case 128: return launch<128>(tw, tx, tsfw, tsfx, tl2, tz, p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace svdq
