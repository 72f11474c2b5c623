// Bounded waits of kernels whose warps have different roles.
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace cskv {

constexpr long long kRoleWaitCycles = 1LL << 31;  // about a second: a wait gives up

// Waits for the phase of `bar` with this parity.  One role that gives up sets *abort (shared memory),
// which makes every role of the CTA leave its loop.  One function for all sites: their code stays
// short, and the roles' loops in the instruction cache.
static __device__ __noinline__ bool role_wait_slow(uint64_t* bar, uint32_t parity, int* abort, int* st) {
  const long long t0 = clock64();
  do {
    if (mbar_poll(bar, parity)) return true;
    if (*(volatile int*)abort) return false;
  } while (clock64() - t0 < kRoleWaitCycles);
  *(volatile int*)abort = 1;
  flag(st, CSKV_DEV_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool role_wait(uint64_t* bar, uint32_t phase, int* abort, int* st) {
  return mbar_try_wait(bar, phase & 1u) || role_wait_slow(bar, phase & 1u, abort, st);
}
// The same for a whole warp, whose lanes agree on the answer.
__device__ __forceinline__ bool role_wait_warp(uint64_t* bar, uint32_t phase, int* abort, int* st) {
  return __all_sync(0xffffffffu, role_wait(bar, phase, abort, st));
}

}  // namespace cskv
