// wait.cuh -- the bounded mbarrier wait every pipelined kernel of the library uses.
#pragma once

#include <cstdint>

#include "ptx_sm103.cuh"
#include "rec_attn_internal.cuh"

namespace recattn {

// Wait for the phase of `bar` with the given parity.  Gives up (returns false) when
// another role of the CTA has aborted (*abort_flag set), or after limit_ns of global
// time, in which case it records REC_ATTN_ERR_TIMEOUT in the status word and raises
// the CTA's abort flag, so the other roles stop at their next wait instead of hanging.
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                             uint64_t limit_ns) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (ptx::mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (ptx::globaltimer() - t0 > limit_ns) {
      *abort_flag = 1;
      set_status(status, REC_ATTN_ERR_TIMEOUT);
      return false;
    }
  }
}

// The same for a whole warp, whose lanes leave together: at the limit, or when another warp raises the
// abort flag, one lane may give up while the next sees the phase complete, and a warp that splits
// there would meet in no later shuffle or matrix instruction again.
__device__ __forceinline__ bool bounded_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                                  uint64_t limit_ns) {
  const bool ok = bounded_wait(bar, parity, abort_flag, status, limit_ns);
  return __all_sync(0xffffffffu, ok);
}

// Wait for a copy (or matrix instructions) of the thread's own to finish before the CTA reuses what they
// write, or leaves.  Bounded too; it waits in earnest only after an abort.
__device__ __forceinline__ void bounded_drain(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity))
    if (ptx::globaltimer() - t0 > limit_ns) return;
}

}  // namespace recattn
