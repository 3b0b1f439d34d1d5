// What the cache attention kernels that load by TMA have in common: copies of scale bytes, and waits that end.
//
// Every wait has a limit.  The first that runs out sets the block's abort word and the call's status word; from then on
// waits return at once, and the block walks through its share to its end on whatever its memory holds, so that no warp
// is left at a barrier.  The producer stops loading, so a stage is never filled while something may still land in it, and
// waits for the copies that are in flight before the block's shared memory is released.
#pragma once

#include "cache.cuh"
#include "sm100.cuh"

namespace pisa {
namespace cache {

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(sm100::smem_u32(dst)), "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar)) : "memory");
}

// Whether the phase has completed; sm.abort: the block's abort word.  alive: where a warp whose work between two arrivals
// may outlast the limit says when it was last seen at it (nullptr: there is none); the limit counts from there.
template <typename S>
__device__ __forceinline__ bool wait_for(S& sm, uint64_t* bar, uint32_t parity, unsigned long long limit_ns, int* status,
                                         const volatile unsigned long long* alive = nullptr) {
  if (sm100::mbar_try_wait(bar, parity)) return true;
  volatile int* abort = &sm.abort;
  const uint64_t t0 = sm100::globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (sm100::mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if ((it & 63u) == 0u) {
      const uint64_t now = sm100::globaltimer_ns();
      if (now - t0 > limit_ns && (!alive || (long long)(now - *alive) > (long long)limit_ns)) break;
    }
  }
  *abort = 1;
  set_status(status, PISA_DEVERR_WAIT_TIMEOUT);
  return false;
}

template <typename S>
__device__ __forceinline__ bool aborted(const S& sm) { return *reinterpret_cast<const volatile int*>(&sm.abort) != 0; }

}  // namespace cache
}  // namespace pisa
