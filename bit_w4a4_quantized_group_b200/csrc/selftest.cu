// Self-test of the failure path: a bounded wait that is meant to run out.
//
// A cluster of two CTAs of one warp.  CTA 0 waits on an mbarrier that nothing arrives at, half of its
// lanes for a phase that counts as complete: they pass at once, as at a barrier that completes just as
// the others' limit runs out.  The wait gives up after the given time, records kErrSiteSelftest in the
// device error word and says so to every lane (kErrSiteSelftestParted otherwise).  CTA 1 waits for
// nothing, learns of the abort (kErrSiteSelftestPeer otherwise) and keeps its memory for kDrainNs more, like
// the CTAs of every kernel after an abort.  Both return normally, so the context stays usable.
// This exercises, on the device, the waits and the abort path of the library's kernels, without any
// fault or hang.
#include <cuda_runtime.h>
#include <cstdint>

#include "ptx.cuh"
#include "svdq_device.cuh"

namespace svdq {
namespace {

__global__ void __cluster_dims__(2, 1, 1) selftest_bounded_wait_kernel(int* err, uint64_t limit_ns) {
  __shared__ uint64_t bar;
  __shared__ volatile int abort_flag;
  if (threadIdx.x == 0) {
    ptx::mbar_init(&bar, 1);
    abort_flag = 0;
    ptx::fence_mbar_init();
  }
  ptx::cluster_sync();           // both flags are cleared before either is raised
  const bool first = ptx::cluster_ctarank() == 0;
  // phase 0 never completes: no thread arrives; the one before it (parity 1) has
  if (first) {
    if (wait_bounded_warp(&bar, threadIdx.x & 1, &abort_flag, err, kErrSiteSelftest, limit_ns))
      atomicExch(err, kErrSiteSelftestParted);
    else
      leave_aborted(&abort_flag);
  }
  ptx::cluster_sync();
  if (abort_flag == 0) atomicExch(err, kErrSiteSelftestPeer);
}

}  // namespace

cudaError_t launch_selftest_bounded_wait(int* err, uint64_t limit_ns, cudaStream_t s) {
  selftest_bounded_wait_kernel<<<2, 32, 0, s>>>(err, limit_ns);
  return cudaGetLastError();
}

}  // namespace svdq
