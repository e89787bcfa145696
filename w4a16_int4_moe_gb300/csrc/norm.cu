// norm.cu -- the residual's addition and the RMS norm in front of the expert
// layer, with a BF16 and an 8-bit output.
//
//   h = x + residual, y = h * rsqrt(mean(h^2) + eps) * weight, in FP32; the
//   BF16 residual, the BF16 y and the e4m3 y / scale are each rounded once.
//   scale = max(amax |y|, 1e-10) / 448 of a 128-column group or of the row
//   (448 is the largest e4m3 value; the floor keeps the scale a normal number,
//   so that an all-zero group divides to zero).

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace w4a16 {

namespace {

constexpr int kNormThreads = 256;
constexpr float kAmaxFloor = 1e-10f;
constexpr float kE4m3Max = 448.f;

// max that keeps a NaN of either operand
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

}  // namespace

// One CTA per row; the row is read again for each step.
__global__ void __launch_bounds__(kNormThreads) w4a16_add_rms_norm_kernel(const NormArgs a) {
  __shared__ float part[kNormThreads / 32];
  extern __shared__ float y_row[];
  const int row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const __nv_bfloat16* x =
      reinterpret_cast<const __nv_bfloat16*>(a.x) + static_cast<long long>(row) * a.x_stride;
  const __nv_bfloat16* r =
      a.residual == nullptr ? nullptr
                            : reinterpret_cast<const __nv_bfloat16*>(a.residual) +
                                  static_cast<long long>(row) * a.residual_stride;
  const __nv_bfloat16* w = reinterpret_cast<const __nv_bfloat16*>(a.weight);
  const long long at = static_cast<long long>(row) * a.hidden;
  float ss = 0.f;
  for (int c = threadIdx.x; c < a.hidden; c += kNormThreads) {
    float h = __bfloat162float(x[c]);
    if (r != nullptr) {
      h += __bfloat162float(r[c]);
      reinterpret_cast<__nv_bfloat16*>(a.residual_out)[at + c] = __float2bfloat16_rn(h);
    }
    y_row[c] = h;
    ss += h * h;
  }
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) part[warp] = ss;
  __syncthreads();
  ss = 0.f;
  for (int i = 0; i < kNormThreads / 32; ++i) ss += part[i];
  const float inv = rsqrtf(ss / static_cast<float>(a.hidden) + a.eps);
  for (int c = threadIdx.x; c < a.hidden; c += kNormThreads) {
    const float y = y_row[c] * inv * __bfloat162float(w[c]);
    y_row[c] = y;
    if (a.out != nullptr) reinterpret_cast<__nv_bfloat16*>(a.out)[at + c] = __float2bfloat16_rn(y);
  }
  if (a.fp8_group == W4A16_FP8_NONE) return;
  __syncthreads();
  const int group = a.fp8_group == W4A16_FP8_ROW ? a.hidden : a.fp8_group;
  const int groups = (a.hidden + group - 1) / group;
  for (int g = warp; g < groups; g += kNormThreads / 32) {
    const int end = min(a.hidden, (g + 1) * group);
    float amax = kAmaxFloor;
    for (int c = g * group + lane; c < end; c += 32) amax = max_nan(amax, fabsf(y_row[c]));
    for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float scale = amax / kE4m3Max;
    if (lane == 0) a.scales[static_cast<long long>(row) * groups + g] = scale;
    for (int c = g * group + lane; c < end; c += 32)
      a.out_fp8[at + c] = __nv_cvt_float_to_fp8(y_row[c] / scale, __NV_SATFINITE, __NV_E4M3);
  }
}

cudaError_t launch_add_rms_norm(const NormArgs& args, int sms, cudaStream_t stream) {
  (void)sms;
  const size_t smem = static_cast<size_t>(args.hidden) * sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(w4a16_add_rms_norm_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kNormMaxHidden * static_cast<int>(sizeof(float)));
  if (e != cudaSuccess) return e;
  w4a16_add_rms_norm_kernel<<<args.rows, kNormThreads, smem, stream>>>(args);
  return cudaGetLastError();
}

}  // namespace w4a16
