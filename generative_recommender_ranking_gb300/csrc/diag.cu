// diag.cu -- self-check of the bounded waits the attention kernels use: one CTA waits on
// an mbarrier that nothing ever arrives at, so the wait must give up after its limit,
// record REC_ATTN_ERR_TIMEOUT in a status word and return, leaving the context usable.
#include <cuda_runtime.h>

#include "launchers.cuh"
#include "wait.cuh"

namespace recattn {

namespace {

__global__ void k_wait_timeout(int* status, unsigned long long limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    ptx::mbar_init(&bar, 1);
    abort_flag = 0;
    ptx::fence_barrier_init();
  }
  __syncthreads();
  // no arrival ever comes: a whole warp waits, and one lane of another
  if (threadIdx.x < 32) bounded_wait_warp(&bar, 0, &abort_flag, status, limit_ns);
  else if (threadIdx.x == 32) bounded_wait(&bar, 0, &abort_flag, status, limit_ns);
}

}  // namespace

cudaError_t launch_wait_timeout(int* status, unsigned long long limit_ns, cudaStream_t st) {
  k_wait_timeout<<<1, 64, 0, st>>>(status, limit_ns);
  return cudaGetLastError();
}

}  // namespace recattn
