// pipe.cuh -- rings of slots between the warps of a CTA or a cluster: positions,
// and waits that end.
#pragma once

#include "ptx.cuh"

namespace w4a16 {

namespace {

// A wait gives up after `limit` cycles, or once another one of the CTA has.
__device__ __forceinline__ bool give_up(volatile int* failed, long long t0, long long limit) {
  if (*failed) return true;
  if (clock64() - t0 <= limit) return false;
  *failed = 1;
  return true;
}
template <bool kRemote>
__device__ __forceinline__ bool phase_done(uint32_t bar, uint32_t parity) {
  return kRemote ? mbar_try_wait_cluster_now(bar, parity) : mbar_try_wait(bar, parity);
}
// kRemote: threads of other CTAs of the cluster arrive as well. kLook: looks first without
// being suspended (which takes up to some thousand cycles), so that a limit of a
// cycle ends every wait that is not over already; 2 % of a kernel whose waits are short.
template <bool kRemote, bool kLook = false>
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, volatile int* failed,
                                          long long limit) {
  if (kLook ? mbar_test_wait(bar, parity) : phase_done<kRemote>(bar, parity)) return true;
  const long long t0 = clock64();
  while (!give_up(failed, t0, limit))
    if (phase_done<kRemote>(bar, parity)) return true;
  return false;
}

// What a CTA has in flight (copies into its shared memory, MMAs that read it) is
// over before the CTA ends, also where other waits gave up: this one has a bound of
// its own, about a second.
constexpr long long kDrainCycles = 2000000000LL;
template <bool kRemote>
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!phase_done<kRemote>(bar, parity) && clock64() - t0 <= kDrainCycles) {
  }
}

// A position in a ring of slots.
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int slots) {
    if (++slot == slots) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

}  // namespace

}  // namespace w4a16
