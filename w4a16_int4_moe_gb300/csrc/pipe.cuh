// pipe.cuh -- rings of slots between the warps of a CTA or a cluster: positions,
// and waits that end.
#pragma once

#include "ptx.cuh"

namespace w4a16 {

namespace {

constexpr long long kGiveUpCycles = 4000000000LL;  // about two seconds

__device__ __forceinline__ bool give_up(volatile int* failed, long long t0) {
  if (*failed) return true;
  if (clock64() - t0 <= kGiveUpCycles) return false;
  *failed = 1;
  return true;
}
// kRemote: threads of other CTAs of the cluster arrive as well.
template <bool kRemote>
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, volatile int* failed) {
  const auto done = [&] {
    return kRemote ? mbar_try_wait_cluster_now(bar, parity) : mbar_try_wait(bar, parity);
  };
  if (done()) return true;
  const long long t0 = clock64();
  while (!done())
    if (give_up(failed, t0)) return false;
  return true;
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
