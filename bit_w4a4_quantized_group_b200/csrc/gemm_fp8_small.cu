// FP8 GEMM for few tokens (sm_100a): the same product as gemm_fp8.cu with the operands' roles
// exchanged.
//
// With few tokens the work is reading the weights once.  A 256-row tile of tokens would be nearly
// empty and leave too few tiles for the SMs, so here the weights are the 128-row operand of the MMA
// and the tokens its N side, T = 16, 32, 64 or 128 wide: D[n][m] = sum_k W[n][k] X[m][k].  The K
// steps of a tile are split over a cluster of up to 8 CTAs, so that most SMs stream weights at once
// (one CTA per SM).  Each CTA sends its fp32 partial sums to the CTA that owns the tokens, one bulk
// copy through distributed shared memory per receiver; the owner adds them in CTA order
// (deterministic) and the bias before the one rounding to bf16.
//
// Scales: as in gemm_fp8.cu a 512-byte block serves four K steps and has a ring of its own; a CTA
// whose share starts inside such a block loads that block with its first step.
//
// What bounds it: reading the weights, and the 4 us around that.  1 x 3072 x 9216 (M x K x N, here and below)
// takes 7.0 us with its 28 MB of weights in L2 and 8.1 with weights from HBM, which need 4.4; 64 x 3072 x
// 12288 10.9 and 11.5, where 5.9 would do: 96 tiles leave no second CTA for each, so that K is not split and
// 52 SMs have no work.
#include <cuda.h>
#include <cuda_bf16.h>
#include <atomic>
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
constexpr int kMaxSplit = 8;                  // portable cluster size

template <int T>
struct Cfg {
  static constexpr uint32_t kXBytes = T * 128;
  static constexpr uint32_t kStageBytes = kWBytes + kXBytes;
  static constexpr int kStages = T == 16 ? 10 : T == 32 ? 8 : T == 64 ? 7 : 4;       // at most
  static constexpr int kMinStages = T == 16 ? 4 : T == 32 ? 4 : T == 64 ? 3 : 2;     // ... whose ring holds T * 512 bytes
  // partial sums that the cluster's CTAs send here: [CTA][a CTA's share of the tokens][128]
  static constexpr uint32_t kRedBytes = (T + kMaxSplit - 1) * kRowsW * 4;
  static_assert(T * kRowsW * 4 <= kMinStages * kStageBytes, "a CTA's own partial tile lies in its drained ring");
  static constexpr uint32_t kTmemSf0 = T;
  static constexpr uint32_t kTmemCols = T <= 32 ? 64 : T == 64 ? 128 : 256;
  static_assert(T + kSfBufs * 8 <= kTmemCols, "TMEM");
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
  uint64_t sf_full[kSfBufs];     // scale slot holds the weights' and the tokens' block
  uint64_t sf_ready[kSfBufs];    // ... and so does the TMEM buffer of the same number
  uint64_t sf_free[kSfBufs];     // the MMAs that read the TMEM buffer have completed
  uint64_t acc_full;
  uint64_t red_full;             // the other CTAs' partial sums of this CTA's tokens have arrived
  uint32_t tmem_base;
  int abort_flag;
};

template <int T>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp8_small_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                          const __grid_constant__ CUtensorMap tmap_sfw, const __grid_constant__ CUtensorMap tmap_sfx,
                          const __grid_constant__ CUtensorMap tmap_l2, const __grid_constant__ CUtensorMap tmap_z,
                          GemmParams p) {
  using C = Cfg<T>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stages = p.stages;
  uint8_t* sf_smem = smem + stages * C::kStageBytes;
  float* red = reinterpret_cast<float*>(sf_smem + kSfBufs * 2 * kSfBlk);
  SharedTail<T>* sh = reinterpret_cast<SharedTail<T>*>(sf_smem + kSfBufs * 2 * kSfBlk + C::kRedBytes);
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
  // K split: CTA r adds up the tokens [r share, r share + own) of the tile
  const int share = (ntok + ks - 1) / ks;
  const int own = max(0, min(share, ntok - split * share));

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(&sh->full[s], 1);
      ptx::mbar_init(&sh->empty[s], 1);
    }
    for (int b = 0; b < kSfBufs; ++b) {
      ptx::mbar_init(&sh->sf_full[b], 1);
      ptx::mbar_init(&sh->sf_ready[b], 1);
      ptx::mbar_init(&sh->sf_free[b], 1);
    }
    ptx::mbar_init(&sh->acc_full, 1);
    ptx::mbar_init(&sh->red_full, 1);
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
  if (ks > 1) {
    if (threadIdx.x == 0)
      ptx::mbar_arrive_expect_tx(&sh->red_full, static_cast<uint32_t>((ks - 1) * own * kRowsW * 4));
    ptx::cluster_arrive();                // waited for before anything is sent: every CTA has started
  }
  const uint32_t tmem = sh->tmem_base;
  ptx::griddep_launch_dependents();
  // the set-up above may overlap the end of the kernel that writes X and Z
  ptx::griddep_wait();
  // this thread's four columns of the bias, on their way while the weights stream
  const int col = 4 * lane;
  uint2 braw = make_uint2(0u, 0u);
  if (p.bias) braw = __ldg(reinterpret_cast<const uint2*>(p.bias + n0 + col));

  // step k < nk of this CTA is the weights' K step kb + k; its first step, and each one that is a
  // multiple of four, starts a scale block
  auto starts_block = [&](int k) { return k < nk && (k == 0 || ((kb + k) & 3) == 0); };

  if (warp == kProdWarp) {
    if (lane == 0) {
      ptx::prefetch_tmap(&tmap_w);
      ptx::prefetch_tmap(&tmap_x);
      int s = 0, b = 0;
      uint32_t ph = 1, sfph = 1;
      for (int k = 0; k < nk + nk_lr; ++k) {
        if (!wait_bounded_call(&sh->empty[s], ph, abort_flag, p.err, kErrSiteGemmEmpty)) break;
        if (starts_block(k)) {
          if (!wait_bounded_call(&sh->sf_free[b], sfph, abort_flag, p.err, kErrSiteGemmSfFree)) break;
          uint8_t* sf = sf_smem + b * 2 * kSfBlk;
          ptx::mbar_arrive_expect_tx(&sh->sf_full[b], 2 * kSfBlk);
          ptx::tma_load_3d(sf, &tmap_sfw, &sh->sf_full[b], 0, (kb + k) >> 2, n0 >> 7);
          ptx::tma_load_3d(sf + kSfBlk, &tmap_sfx, &sh->sf_full[b], 0, (kb + k) >> 2, m0 >> 7);
          if (++b == kSfBufs) { b = 0; sfph ^= 1u; }
        }
        uint8_t* st = smem + s * C::kStageBytes;
        ptx::mbar_arrive_expect_tx(&sh->full[s], C::kStageBytes);
        if (k < nk) {
          ptx::tma_load_3d(st, &tmap_w, &sh->full[s], 0, n0, kb + k);
          ptx::tma_load_3d(st + kWBytes, &tmap_x, &sh->full[s], 0, m0, kb + k);
        } else {
          ptx::tma_load_2d(st, &tmap_l2, &sh->full[s], (k - nk) * 64, n0);
          ptx::tma_load_2d(st + kWBytes, &tmap_z, &sh->full[s], (k - nk) * 64, m0);
        }
        if (++s == stages) { s = 0; ph ^= 1u; }
      }
    }
    __syncwarp();
    end_issuing_role(abort_flag);
  } else if (warp == kCopyWarp) {
    // scale slot b -> TMEM buffer b; the producer refills the slot when the buffer is free
    int b = 0;
    uint32_t sfph = 0;
    const uint64_t sfdesc0 = ptx::sdesc_sf(ptx::smem_u32(sf_smem));
    const int blocks = ((kb + nk - 1) >> 2) - (kb >> 2) + 1;
    for (int i = 0; i < blocks; ++i) {
      if (!wait_bounded_call_warp(&sh->sf_full[b], sfph, abort_flag, p.err, kErrSiteGemmFull)) break;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        const uint64_t sd = sfdesc0 + static_cast<uint64_t>(b) * (2 * kSfBlk / 16);
        const uint32_t sfa = tmem + C::kTmemSf0 + static_cast<uint32_t>(b) * 8;
        ptx::tmem_cp_32x128b_warpx4(sfa, sd);
        ptx::tmem_cp_32x128b_warpx4(sfa + 4, sd + kSfBlk / 16);
        ptx::tc_commit(&sh->sf_ready[b]);
      }
      __syncwarp();
      if (++b == kSfBufs) { b = 0; sfph ^= 1u; }
    }
    end_issuing_role(abort_flag);
  } else if (warp == kMmaWarp) {
    int s = 0, b = 0;
    uint32_t ph = 0, sfph = 0;
    const uint32_t id16 = idesc_bf16(kRowsW, T);
    const uint64_t desc0 = ptx::sdesc_sw128(ptx::smem_u32(smem));
    for (int k = 0; k < nk + nk_lr; ++k) {
      if (!wait_bounded_call_warp(&sh->full[s], ph, abort_flag, p.err, kErrSiteGemmFull)) break;
      const bool main_step = k < nk;
      const uint32_t id = static_cast<uint32_t>((kb + k) & 3);
      if (starts_block(k) && !wait_bounded_call_warp(&sh->sf_ready[b], sfph, abort_flag, p.err, kErrSiteGemmSfReady)) break;
      ptx::tc_fence_after();
      const bool sf_done = main_step && (id == 3 || k == nk - 1);
      if (ptx::elect_one()) {
        const uint64_t wd = desc0 + static_cast<uint64_t>(s) * (C::kStageBytes / 16);
        const uint64_t xd = wd + kWBytes / 16;
        if (main_step) {
          const uint32_t sfa = tmem + C::kTmemSf0 + static_cast<uint32_t>(b) * 8;
          const uint32_t sfb = sfa + 4;      // the tile starts its scale block: m0 is 0, or a multiple of 128 with T = 128
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
      if (++s == stages) { s = 0; ph ^= 1u; }
    }
    end_issuing_role(abort_flag);
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------ thread = weight row, column = token
    const int q = warp & 3;
    const int n = q * 32 + lane;
    if (ks > 1) ptx::cluster_wait();
    if (wait_bounded_call_warp(&sh->acc_full, 0u, abort_flag, p.err, kErrSiteGemmAccFull)) {
      ptx::tc_fence_after();
      const uint32_t base = tmem + (static_cast<uint32_t>(q * 32) << 16);
      float* part = reinterpret_cast<float*>(smem) + n;       // [token][128], in the drained ring
      constexpr int kCols = T < 32 ? T : 32;
#pragma unroll 1
      for (int c = 0; c < ntok; c += kCols) {
        uint32_t v[kCols];
#pragma unroll
        for (int h = 0; h < kCols; h += 16)
          ptx::tmem_ld_32x32b_x16(base + c + h, *reinterpret_cast<uint32_t(*)[16]>(v + h));
        ptx::tmem_wait_ld();
        // whole chunks: rows past the last token stay inside the T rows of the tile
#pragma unroll
        for (int e = 0; e < kCols; ++e)
          if (SVDQ_IN_SMEM(smem_raw, part + (c + e) * kRowsW, 4, p.err))
            part[(c + e) * kRowsW] = __uint_as_float(v[e]);
      }
      ptx::tc_fence_before();
    } else {
      leave_aborted(abort_flag);
    }
    if (ks > 1) {
      // every other CTA gets its tokens' rows with one bulk copy
      ptx::fence_proxy_async_smem();
      named_barrier_sync(1, 128);
      if (warp == kEpiWarp0 && lane < ks && lane != split && *abort_flag == 0) {
        const int rows = min(share, ntok - lane * share);
        if (rows > 0)
          ptx::bulk_copy_to_cta(ptx::mapa_shared(ptx::smem_u32(red + split * share * kRowsW), static_cast<uint32_t>(lane)),
                                reinterpret_cast<const float*>(smem) + lane * share * kRowsW,
                                static_cast<uint32_t>(rows * kRowsW * 4),
                                ptx::mapa_shared(ptx::smem_u32(&sh->red_full), static_cast<uint32_t>(lane)));
      }
      __syncwarp();
    }
  }

  if (ks > 1 && warp < kEpiWarp0) ptx::cluster_wait();       // the epilogue warps have waited
  __syncthreads();                                           // this CTA's own rows lie in its ring
  bool ok = *abort_flag == 0;
  if (ks > 1) {
    if (!wait_bounded_call_warp(&sh->red_full, 0u, abort_flag, p.err, kErrSiteGemmAccFinal)) {
      ok = false;
      leave_aborted(abort_flag);
    }
    // what the others sent has arrived; when all CTAs say so, every copy has left its source
    __syncwarp();
    ptx::cluster_arrive();
  }
  // The partial sums are added in CTA order; a warp takes a token, a thread four columns.
  if (ok) {
    const float4 b = make_float4(__uint_as_float(braw.x << 16), __uint_as_float(braw.x & 0xFFFF0000u),
                                 __uint_as_float(braw.y << 16), __uint_as_float(braw.y & 0xFFFF0000u));
    const float* mine = reinterpret_cast<const float*>(smem) + split * share * kRowsW + col;
#pragma unroll 1
    for (int i = warp; i < own; i += kThreads / 32) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int r = 0; r < ks; ++r) {
        const float* src = r == split ? mine + i * kRowsW : red + (r * share + i) * kRowsW + col;
        if (!SVDQ_IN_SMEM(smem_raw, src, 16, p.err)) continue;
        const float4 v = *reinterpret_cast<const float4*>(src);
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
      const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x + b.x, a.y + b.y), hi = __floats2bfloat162_rn(a.z + b.z, a.w + b.w);
      if (SVDQ_IN_GLOBAL(n0 + col + 4 <= p.N, p.err))
        *reinterpret_cast<uint2*>(p.Y + static_cast<size_t>(m0 + split * share + i) * p.N + n0 + col) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
  }
  __syncwarp();
  if (ks > 1) ptx::cluster_wait();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int T>
constexpr size_t smem_bytes(int stages = Cfg<T>::kStages) {
  return 1024 + stages * Cfg<T>::kStageBytes + kSfBufs * 2 * kSfBlk + Cfg<T>::kRedBytes + sizeof(SharedTail<T>);
}

template <int T>
void fill_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], int clusters, int ks, int stages,
                 cudaStream_t s) {
  cfg.gridDim = dim3(static_cast<unsigned>(clusters) * static_cast<unsigned>(ks), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem_bytes<T>(stages);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // may start under the kernel before
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
}

// Clusters of ks CTAs that the current device holds at once (0 on error), asked once per device.
template <int T>
int resident_clusters(int ks) {
  static std::atomic<int> cache[64][kMaxSplit + 1];      // 0: not asked yet, else 1 + the figure
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int known = cache[dev][ks].load(std::memory_order_relaxed);
  if (known > 0) return known - 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  fill_config<T>(cfg, attr, 1, ks, Cfg<T>::kStages, nullptr);
  cfg.numAttrs = 1;                                      // the cluster alone
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, gemm_fp8_small_kernel<T>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  cache[dev][ks].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <int T>
cudaError_t launch(const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& tsfw, const CUtensorMap& tsfx,
                   const CUtensorMap& tl2, const CUtensorMap& tz, GemmParams p, cudaStream_t s, int* ksplit) {
  static_assert(smem_bytes<T>() <= 232448, "shared memory of one CTA");
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(gemm_fp8_small_kernel<T>), smem_bytes<T>());
  if (e != cudaSuccess) return e;
  // The widest split with every cluster resident at once: a second wave costs a whole pass.
  const int nk = p.K / kKTile;
  p.ksplit = 1;
  for (int ks = nk < kMaxSplit ? nk : kMaxSplit; ks > 1; --ks)
    if (resident_clusters<T>(ks) >= p.num_tiles) {
      p.ksplit = ks;
      break;
    }
  *ksplit = p.ksplit;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  // A ring no longer than a CTA's steps, and no deeper than 12 MB in flight over all CTAs need (1.5 us
  // of latency at 8 TB/s): a smaller CTA leaves the next launch room to set itself up.
  const int steps = (nk + p.ksplit - 1) / p.ksplit + (p.rank + 63) / 64;
  const int64_t deep = (int64_t(12) << 20) / (int64_t(p.num_tiles) * p.ksplit * Cfg<T>::kStageBytes) + 1;
  p.stages = steps < deep ? steps : static_cast<int>(deep);
  if (p.stages < Cfg<T>::kMinStages) p.stages = Cfg<T>::kMinStages;
  if (p.stages > Cfg<T>::kStages) p.stages = Cfg<T>::kStages;
  fill_config<T>(cfg, attr, p.num_tiles, p.ksplit, p.stages, s);
  e = cudaLaunchKernelEx(&cfg, gemm_fp8_small_kernel<T>, tw, tx, tsfw, tsfx, tl2, tz, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

int gemm_fp8_small_tokens(int M, int N, int K, int num_sms, float other_us) {
  // Up to 64 tokens this kernel is the faster one (1 x 3072 x 9216: 7.7 us against 12; 64 x 3072 x 12288:
  // 12.4 against 14).  Beyond, tiles of 128 tokens pay where the other kernel has few
  // tiles and a long K: 4.3 us and 25 ns per token of a tile to start, add up and drain, and per K step 0.22 us or the time of
  // 32 KB for every CTA at 8.6 TB/s (us measured, this kernel / the other: 128 x 12288 x 3072 15.9 / 26,
  // 512 x 8192 x 512 10.9 / 19, 512 x 3072 x 9216 42 / 17).
  if (M <= 64) return M <= 16 ? 16 : M <= 32 ? 32 : 64;
  const int64_t tiles = int64_t(N / kRowsW) * ((M + 127) / 128);
  const int nk = K / kKTile;
  int64_t ks = num_sms / tiles;
  if (ks > kMaxSplit) ks = kMaxSplit;
  if (ks > nk) ks = nk;
  if (ks < 1) ks = 1;
  const int64_t ctas = tiles * ks, waves = (ctas + num_sms - 1) / num_sms;
  const float step = 0.0038f * static_cast<float>(ctas < num_sms ? ctas : num_sms);
  const float us = 4.3f + 0.025f * static_cast<float>(M < 128 ? M : 128) + static_cast<float>(waves * ((nk + ks - 1) / ks)) * (step > 0.22f ? step : 0.22f);
  return us < other_us ? 128 : 0;
}

cudaError_t launch_gemm_fp8_small(int tokens, const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& tsfw,
                                  const CUtensorMap& tsfx, const CUtensorMap& tl2, const CUtensorMap& tz,
                                  const GemmParams& p, cudaStream_t s, int* ksplit) {
  switch (tokens) {
    case 16: return launch<16>(tw, tx, tsfw, tsfx, tl2, tz, p, s, ksplit);
    case 32: return launch<32>(tw, tx, tsfw, tsfx, tl2, tz, p, s, ksplit);
    case 64: return launch<64>(tw, tx, tsfw, tsfx, tl2, tz, p, s, ksplit);
    case 128: return launch<128>(tw, tx, tsfw, tsfx, tl2, tz, p, s, ksplit);
  }
  return cudaErrorInvalidValue;
}

}  // namespace svdq
