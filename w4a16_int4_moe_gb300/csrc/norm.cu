// norm.cu -- the residual's addition and the RMS norm in front of the expert
// layer, with a BF16 and an 8-bit output.
//
//   h = x + residual, y = h * rsqrt(mean(h^2) + eps) * weight, in FP32; the
//   BF16 residual, the BF16 y and the e4m3 y / scale are each rounded once.
//   scale = max(amax |y|, 1e-10) / 448 of a 128-column group or of the row
//   (448 is the largest e4m3 value; the floor keeps the scale a normal number,
//   so that an all-zero group divides to zero; a group or row with an infinity
//   or a NaN has a NaN scale and NaN codes).
//
// Bound by memory for many rows, by latency for few: 8192 rows of 7168 with a
// residual, BF16 and 8-bit outputs and group scales take 79 us, 6.7 TB/s of the
// 530 MB, which is the copy rate; 576 such rows 9 us (4.1 TB/s), one 2.3, one
// BF16 row 1.9 (in a graph). A row is read once into registers (eight columns a
// thread and chunk: 16-byte loads), its sum of squares joined over the threads
// of the row, and everything is written from registers. A block of 16 lanes
// holds the 128 columns of a group of the 8-bit form, so a group's largest
// value needs four shuffles and no shared memory.

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace w4a16 {

namespace {

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

}  // namespace

// One row per CTA of kThreads threads; chunk c of thread t holds the columns
// 8 (c * kThreads + t) .. + 7, kChunks chunks.
template <int kThreads, int kChunks>
__global__ void __launch_bounds__(kThreads) w4a16_add_rms_norm_kernel(const NormArgs a) {
  __shared__ float part[2][kThreads / 32];
  const int row = blockIdx.x;
  const long long at = static_cast<long long>(row) * a.hidden;
  const uint16_t* x = a.x + static_cast<long long>(row) * a.x_stride;
  float h[kChunks][8];
  uint4 w[kChunks];
  grid_dependency_wait();
  grid_dependents_go();
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int k = 8 * (c * kThreads + static_cast<int>(threadIdx.x));
    w[c] = make_uint4(0u, 0u, 0u, 0u);
    if (k < a.hidden) w[c] = __ldg(reinterpret_cast<const uint4*>(a.weight + k));
  }
  uint4 in[kChunks], res[kChunks];
  const uint16_t* r = a.residual == nullptr
                          ? nullptr
                          : a.residual + static_cast<long long>(row) * a.residual_stride;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int k = 8 * (c * kThreads + static_cast<int>(threadIdx.x));
    in[c] = res[c] = make_uint4(0u, 0u, 0u, 0u);
    if (k < a.hidden) {
      in[c] = *reinterpret_cast<const uint4*>(x + k);
      if (r != nullptr) res[c] = *reinterpret_cast<const uint4*>(r + k);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    unpack8(in[c], h[c]);
    if (r != nullptr) {
      float f[8];
      unpack8(res[c], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] += f[i];
      const int k = 8 * (c * kThreads + static_cast<int>(threadIdx.x));
      if (k < a.hidden) *reinterpret_cast<uint4*>(a.residual_out + at + k) = pack8(h[c]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(h[c][i], h[c][i], ss);
  }
  ss = row_join<kThreads>(ss, part[0], [](float p, float q) { return p + q; });
  const float inv = rsqrtf(ss / static_cast<float>(a.hidden) + a.eps);
  float amax = kAmaxFloor;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int k = 8 * (c * kThreads + static_cast<int>(threadIdx.x));
    float f[8];
    unpack8(w[c], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[c][i] = h[c][i] * inv * f[i];
    if (a.out != nullptr && k < a.hidden) *reinterpret_cast<uint4*>(a.out + at + k) = pack8(h[c]);
    if (a.fp8_group == W4A16_FP8_NONE) continue;
    // (columns past the row are 0, or NaN in a row that has a NaN norm)
    float top = kAmaxFloor;
    if (k < a.hidden) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(h[c][i]));
    }
    if (a.fp8_group == W4A16_FP8_ROW) {
      amax = max_nan(amax, top);
      continue;
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float scale = group_scale(top);
    if (k < a.hidden) {
      *reinterpret_cast<uint2*>(a.out_fp8 + at + k) = codes8(h[c], scale);
      if ((threadIdx.x & 15) == 0)
        a.scales[static_cast<long long>(row) * ((a.hidden + 127) / 128) + k / 128] = scale;
    }
  }
  if (a.fp8_group != W4A16_FP8_ROW) return;
  amax = row_join<kThreads>(amax, part[1], [](float p, float q) { return max_nan(p, q); });
  const float scale = group_scale(amax);
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int k = 8 * (c * kThreads + static_cast<int>(threadIdx.x));
    if (k < a.hidden) *reinterpret_cast<uint2*>(a.out_fp8 + at + k) = codes8(h[c], scale);
  }
  if (threadIdx.x == 0) a.scales[row] = scale;
}

// Threads and chunks of a row. With at most a row an SM, more threads and fewer
// chunks: a row of 7168 takes 2.2 us on 512 x 2 and 2.7 on 256 x 4 (with group
// scales). With more rows as few threads' registers without columns as can be,
// in CTAs of 128 or 256: 8192 rows of 2088 take 21 us on 128 x 3 and 27 on
// 384 x 1 or 256 x 2, 8192 of 7168 79 us on 256 x 4 and 88 on 512 x 2; up to
// four rows an SM the former's CTAs fit at once and 384 x 1 is faster (576 rows
// of 2088: 2.4 and 2.7 us).
cudaError_t launch_add_rms_norm(const NormArgs& args, int sms, cudaStream_t stream) {
  const int need = (args.hidden + 7) / 8;  // threads of one chunk
  const auto run = [&](void (*kernel)(NormArgs), int threads) {
    return launch_dependent(kernel, args.rows, threads, 0, 1, stream, args);
  };
  if (need <= 32) return run(w4a16_add_rms_norm_kernel<32, 1>, 32);
  if (need <= 128) return run(w4a16_add_rms_norm_kernel<128, 1>, 128);
  if (need <= 256) return run(w4a16_add_rms_norm_kernel<256, 1>, 256);
  if (need <= 384 && args.rows <= 4 * sms) return run(w4a16_add_rms_norm_kernel<384, 1>, 384);
  if (need <= 384) return run(w4a16_add_rms_norm_kernel<128, 3>, 128);
  if (need <= 512) return run(w4a16_add_rms_norm_kernel<256, 2>, 256);
  if (need <= 1024 && args.rows <= sms) return run(w4a16_add_rms_norm_kernel<512, 2>, 512);
  if (need <= 768) return run(w4a16_add_rms_norm_kernel<256, 3>, 256);
  if (need <= 1024) return run(w4a16_add_rms_norm_kernel<256, 4>, 256);
  if (args.rows <= sms) return run(w4a16_add_rms_norm_kernel<512, 4>, 512);
  if (need <= 1280) return run(w4a16_add_rms_norm_kernel<256, 5>, 256);
  if (need <= 1536) return run(w4a16_add_rms_norm_kernel<256, 6>, 256);
  return run(w4a16_add_rms_norm_kernel<512, 4>, 512);
}

}  // namespace w4a16
