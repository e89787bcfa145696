// norm_row.cuh -- a row of a norm in the registers of a CTA's threads: eight
// columns a thread and chunk, joins over the row, the 8-bit form.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace w4a16 {

constexpr float kAmaxFloor = 1e-10f;
constexpr float kE4m3Max = 448.f;

// max that keeps a NaN of either operand
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The scale of a group or row with this amax: NaN also beside an infinity
// (infinity * 0), whose finite neighbours would become zeros that decode to NaN.
__device__ __forceinline__ float group_scale(float amax) {
  return __fdiv_rn(fmaf(amax, 0.f, amax), kE4m3Max);
}

// eight values times the scale's reciprocal, rounded to e4m3 (the product is
// off the quotient by at most one FP32 step, which moves a code only where the
// quotient lies that near to a border; eight divisions cost the bandwidth:
// 94 us for 8192 rows of 7168)
__device__ __forceinline__ uint2 codes8(const float (&y)[8], float scale) {
  const float r = __fdiv_rn(1.f, scale);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(y[4 * i] * r, y[4 * i + 1] * r), __NV_SATFINITE,
        __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(y[4 * i + 2] * r, y[4 * i + 3] * r),
        __NV_SATFINITE, __NV_E4M3);
    w[i] = static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
  }
  return make_uint2(w[0], w[1]);
}

// Joins a value over the kThreads threads of a row (all of the CTA).
template <int kThreads, typename Op>
__device__ __forceinline__ float row_join(float v, float* part, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if constexpr (kThreads > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) v = op(v, part[i]);
  }
  return v;
}

}  // namespace w4a16
