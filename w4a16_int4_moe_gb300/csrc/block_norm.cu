// block_norm.cu -- the norms after and before a block, with the block's gate and
// scales and the residual:
//
//   p = x * rsqrt(mean(x^2) + eps) * (post + offset)   (p = x without post)
//   h = residual_scale * residual + branch_scale * gate * p
//   y = h * rsqrt(mean(h^2) + eps) * (pre + offset)
//
// The simplest form that is right for every case: a CTA has a row and goes over
// it again for each of the three steps.

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace w4a16 {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float from_bf16(uint16_t v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
__device__ __forceinline__ uint16_t to_bf16(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&b);
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename Op>
__device__ __forceinline__ float row_join(float v, float* part, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) v = op(v, part[i]);
  return v;
}

}  // namespace

__global__ void __launch_bounds__(kThreads) w4a16_block_norm_kernel(const BlockNormArgs a) {
  extern __shared__ float hs[];  // the row's h, then y
  __shared__ float part[kThreads / 32];
  const long long row = blockIdx.x;
  const int tid = threadIdx.x, n = a.hidden;
  const auto add = [](float p, float q) { return p + q; };
  const auto most = [](float p, float q) { return max_nan(p, q); };
  grid_dependency_wait();
  grid_dependents_go();
  const auto x_at = [&](int c) {
    return a.x_f32 ? static_cast<const float*>(a.x)[row * a.x_stride + c]
                   : from_bf16(static_cast<const uint16_t*>(a.x)[row * a.x_stride + c]);
  };
  float inv = 1.f;
  if (a.post_weight != nullptr) {
    float ss = 0.f;
    for (int c = tid; c < n; c += kThreads) ss = fmaf(x_at(c), x_at(c), ss);
    inv = rsqrtf(row_join(ss, part, add) / static_cast<float>(n) + a.eps);
  }
  float ss = 0.f;
  for (int c = tid; c < n; c += kThreads) {
    float p = x_at(c);
    if (a.post_weight != nullptr) p = p * inv * (from_bf16(a.post_weight[c]) + a.weight_offset);
    float h = a.branch_scale * p;
    if (a.gate != nullptr) h *= from_bf16(a.gate[row * a.gate_stride + c]);
    if (a.residual != nullptr)
      h = fmaf(a.residual_scale, from_bf16(a.residual[row * a.residual_stride + c]), h);
    if (a.h_out != nullptr) a.h_out[row * n + c] = to_bf16(h);
    hs[c] = h;
    ss = fmaf(h, h, ss);
  }
  if (a.pre_weight == nullptr) return;
  inv = rsqrtf(row_join(ss, part, add) / static_cast<float>(n) + a.eps);
  float top = 1e-10f;
  for (int c = tid; c < n; c += kThreads) {
    const float y = hs[c] * inv * (from_bf16(a.pre_weight[c]) + a.weight_offset);
    if (a.out != nullptr) a.out[row * n + c] = to_bf16(y);
    hs[c] = y;
    top = max_nan(top, fabsf(y));
  }
  if (a.fp8_group == W4A16_FP8_NONE) return;
  top = row_join(top, part, most);
  const int width = a.fp8_group == W4A16_FP8_ROW ? n : W4A16_FP8_GROUP;
  const int groups = (n + width - 1) / width;
  for (int g = tid >> 5; g < groups; g += kThreads / 32) {
    const int end = min(n, (g + 1) * width);
    float most_of = 1e-10f;
    if (groups > 1)
      for (int c = g * width + (tid & 31); c < end; c += 32) most_of = max_nan(most_of, fabsf(hs[c]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      most_of = max_nan(most_of, __shfl_xor_sync(0xffffffffu, most_of, o));
    if (groups == 1) most_of = top;
    // (NaN also beside an infinity)
    const float scale = __fdiv_rn(fmaf(most_of, 0.f, most_of), 448.f);
    const float r = __fdiv_rn(1.f, scale);
    for (int c = g * width + (tid & 31); c < end; c += 32)
      a.out_fp8[row * n + c] = __nv_cvt_float_to_fp8(hs[c] * r, __NV_SATFINITE, __NV_E4M3);
    if ((tid & 31) == 0) a.scales[row * groups + g] = scale;
  }
}

cudaError_t launch_block_norm(const BlockNormArgs& args, int, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(w4a16_block_norm_kernel,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kNormMaxHidden * 4);
  if (e != cudaSuccess) return e;
  return launch_dependent(w4a16_block_norm_kernel, args.rows, kThreads,
                          static_cast<size_t>(args.hidden) * 4, 1, stream, args);
}

}  // namespace w4a16
