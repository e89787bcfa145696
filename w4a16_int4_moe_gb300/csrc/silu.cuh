// silu.cuh -- the gated products' way out.
#pragma once

namespace w4a16 {

namespace {

// silu(gate) * up = gate / (1 + e^-gate) * up to within 8 steps of FP32 for any finite
// gate. With e = e^(-|gate| / 2) no part of it leaves FP32's range before the result
// does: e^-gate is past it for gates below -88, where silu is -1e-37 and an up may
// be large. (The divisor is 1 to 2, where the quick division is off by two steps.)
__device__ __forceinline__ float silu_times(float gate, float up) {
  const float e = expf(-0.5f * fabsf(gate));
  const float f = gate < 0.f ? e : 1.f;
  return __fdividef(gate * f, fmaf(e, e, 1.f)) * (up * f);
}

// The same from a gate of at least kNearGate, where e^-gate is far inside FP32's range: in
// fewer instructions, and for a result that is rounded to BF16 in half of them, to
// within 2^-16 (the exponential's argument is rounded once, the two approximations are
// off by 2^-22).
constexpr float kNearGate = -80.f;
__device__ __forceinline__ float silu_times_near(float gate, float up) {
  return __fdividef(gate, 1.f + expf(-gate)) * up;
}
__device__ __forceinline__ float silu_times_quick(float gate, float up) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(gate * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return gate * r * up;
}

}  // namespace

}  // namespace w4a16
