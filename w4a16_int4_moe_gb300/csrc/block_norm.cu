// block_norm.cu -- the norms after and before a block, with the block's gate and
// scales and the residual:
//
//   p = x * rsqrt(mean(x^2) + eps) * (post + offset)   (p = x without post)
//   h = residual_scale * residual + branch_scale * gate * p
//   y = h * rsqrt(mean(h^2) + eps) * (pre + offset)
//
// in FP32; the BF16 h, the BF16 y and the e4m3 y / scale are each rounded once.
//
// Bound by memory for many rows, by latency for few. A row is read once into the
// registers of one CTA (eight columns a thread and chunk: 16-byte loads, all
// issued before the first is used), joined twice, and everything is written from
// registers; what keeps the memory busy while a row is joined are the loads of the
// other rows of its SM. 8192 rows of 7168, FP32 x, gates of every token, BF16 and
// 8-bit outputs: 117 us for 765 MB, 6.5 TB/s (0.96 of the copy rate); without
// gates and 8 bits 88 us (0.98); one row 2.6 us (in a graph).

#include <cuda_runtime.h>

#include "internal.h"
#include "norm_row.cuh"
#include "ptx.cuh"

namespace w4a16 {

// One row per CTA of kThreads threads; chunk c of thread t holds the columns
// 8 (c * kThreads + t) .. + 7, kChunks chunks; kCtas rows an SM at least. kX32: x in FP32.
template <bool kX32, int kThreads, int kChunks, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) w4a16_block_norm_kernel(const BlockNormArgs a) {
  __shared__ float part[3][kThreads / 32];
  const long long row = blockIdx.x;
  const auto column = [](int c) { return 8 * (c * kThreads + static_cast<int>(threadIdx.x)); };
  const auto load = [](const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); };
  const auto add = [](float p, float q) { return p + q; };
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  grid_dependency_wait();
  grid_dependents_go();
  float h[kChunks][8];
  uint4 in[kX32 ? 1 : kChunks], res[kChunks], gate[kChunks], w[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int k = column(c);
    const bool inside = k < a.hidden;
    if constexpr (kX32) {
      const float4* x = reinterpret_cast<const float4*>(static_cast<const float*>(a.x) +
                                                        row * a.x_stride + k);
      const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 lo = inside ? x[0] : none, hi = inside ? x[1] : none;
      h[c][0] = lo.x, h[c][1] = lo.y, h[c][2] = lo.z, h[c][3] = lo.w;
      h[c][4] = hi.x, h[c][5] = hi.y, h[c][6] = hi.z, h[c][7] = hi.w;
    } else {
      in[c] = inside ? load(static_cast<const uint16_t*>(a.x) + row * a.x_stride + k) : zero;
    }
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int k = column(c);
    const bool inside = k < a.hidden;
    res[c] =
        inside && a.residual != nullptr ? load(a.residual + row * a.residual_stride + k) : zero;
    gate[c] = inside && a.gate != nullptr ? load(a.gate + row * a.gate_stride + k) : zero;
    w[c] = inside && a.post_weight != nullptr
               ? __ldg(reinterpret_cast<const uint4*>(a.post_weight + k))
               : zero;
  }
  if constexpr (!kX32) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) unpack8(in[c], h[c]);
  }
  if (a.post_weight != nullptr) {
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[c][i], h[c][i], ss);
    ss = row_join<kThreads>(ss, part[0], add);
    const float inv = rsqrtf(ss / static_cast<float>(a.hidden) + a.eps);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float f[8];
      unpack8(w[c], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = h[c][i] * inv * (f[i] + a.weight_offset);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int k = column(c);
    float g[8], r[8];
    unpack8(gate[c], g);
    unpack8(res[c], r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = a.branch_scale * h[c][i];
      if (a.gate != nullptr) v *= g[i];
      if (a.residual != nullptr) v = fmaf(a.residual_scale, r[i], v);
      h[c][i] = v;
    }
    if (k >= a.hidden) {
      // (0 times an infinite factor is NaN)
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = 0.f;
    } else if (a.h_out != nullptr) {
      *reinterpret_cast<uint4*>(a.h_out + row * a.hidden + k) = pack8(h[c]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(h[c][i], h[c][i], ss);
    w[c] = k < a.hidden && a.pre_weight != nullptr
               ? __ldg(reinterpret_cast<const uint4*>(a.pre_weight + k))
               : zero;
  }
  if (a.pre_weight == nullptr) return;
  ss = row_join<kThreads>(ss, part[1], add);
  const float inv = rsqrtf(ss / static_cast<float>(a.hidden) + a.eps);
  float amax = kAmaxFloor;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int k = column(c);
    const bool inside = k < a.hidden;
    float f[8];
    unpack8(w[c], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[c][i] = h[c][i] * inv * (f[i] + a.weight_offset);
    if (a.out != nullptr && inside)
      *reinterpret_cast<uint4*>(a.out + row * a.hidden + k) = pack8(h[c]);
    if (a.fp8_group == W4A16_FP8_NONE) continue;
    // (columns past the row are 0, or NaN in a row that has a NaN norm)
    float top = kAmaxFloor;
    if (inside) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(h[c][i]));
    }
    if (a.fp8_group == W4A16_FP8_ROW) {
      amax = max_nan(amax, top);
      continue;
    }
    // sixteen lanes hold the 128 columns of a group
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float scale = group_scale(top);
    if (inside) {
      *reinterpret_cast<uint2*>(a.out_fp8 + row * a.hidden + k) = codes8(h[c], scale);
      if ((threadIdx.x & 15) == 0) a.scales[row * ((a.hidden + 127) / 128) + k / 128] = scale;
    }
  }
  if (a.fp8_group != W4A16_FP8_ROW) return;
  amax = row_join<kThreads>(amax, part[2], [](float p, float q) { return max_nan(p, q); });
  const float scale = group_scale(amax);
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int k = column(c);
    if (k < a.hidden)
      *reinterpret_cast<uint2*>(a.out_fp8 + row * a.hidden + k) = codes8(h[c], scale);
  }
  if (threadIdx.x == 0) a.scales[row] = scale;
}

namespace {

// Threads and chunks of a row:
//   * up to a row an SM: two chunks of up to 512 threads (152 rows of 7168: 4.3
//     us on 448 x 2, 5.0 on 128 x 7);
//   * more rows: chunks of 128 threads, of seven chunks three such rows an SM (8192
//     rows of 7168: 88 us on 128 x 7, 99 on 448 x 2 or 256 x 4, which are two rows;
//     8192 of 8192: 102 on 128 x 8, 160 on 512 x 2); longer rows 256 x 5 and 256 x 6
//     in 128 registers, two rows an SM (8192 of 12288: 148 us, 203 with one);
//   * of those, rows of up to three chunks take 96 threads where that leaves fewer
//     lanes without columns (8192 rows of 768: 13.4 us on 96 x 1, 15.5 on 128 x 1; of
//     1032 20.4 and 23.6, 1536 24.0 and 26.7, 2088 37.0 and 41.5; 300 to 2000 rows
//     from 6 % less to 2 % more). With more chunks it may cost more than the lanes
//     are worth: 8192 rows of 3840 64.8 and 60.5, of 5376 134 and 92;
//   * behind those 512 x 4, one row an SM (8192 of 16384: 231 us, 256 x 8 256).
template <bool kX32>
cudaError_t launch(const BlockNormArgs& args, int sms, cudaStream_t stream) {
  const int need = (args.hidden + 7) / 8;  // threads of one chunk
  const auto run = [&](void (*kernel)(BlockNormArgs), int threads) {
    return launch_dependent(kernel, args.rows, threads, 0, 1, stream, args);
  };
  if (need <= 32) return run(w4a16_block_norm_kernel<kX32, 32, 1, 1>, 32);
  if (args.rows > sms && need <= 96) return run(w4a16_block_norm_kernel<kX32, 96, 1, 1>, 96);
  if (need <= 128) return run(w4a16_block_norm_kernel<kX32, 128, 1, 1>, 128);
  if (args.rows <= sms) {
    if (need <= 256) return run(w4a16_block_norm_kernel<kX32, 256, 1, 1>, 256);
    if (need <= 384) return run(w4a16_block_norm_kernel<kX32, 384, 1, 1>, 384);
    if (need <= 512) return run(w4a16_block_norm_kernel<kX32, 256, 2, 1>, 256);
    if (need <= 640) return run(w4a16_block_norm_kernel<kX32, 320, 2, 1>, 320);
    if (need <= 768) return run(w4a16_block_norm_kernel<kX32, 384, 2, 1>, 384);
    if (need <= 896) return run(w4a16_block_norm_kernel<kX32, 448, 2, 1>, 448);
    if (need <= 1024) return run(w4a16_block_norm_kernel<kX32, 512, 2, 1>, 512);
  } else {
    if (need <= 192) return run(w4a16_block_norm_kernel<kX32, 96, 2, 1>, 96);
    if (need <= 256) return run(w4a16_block_norm_kernel<kX32, 128, 2, 1>, 128);
    if (need <= 288) return run(w4a16_block_norm_kernel<kX32, 96, 3, 1>, 96);
    if (need <= 384) return run(w4a16_block_norm_kernel<kX32, 128, 3, 1>, 128);
    if (need <= 512) return run(w4a16_block_norm_kernel<kX32, 128, 4, 1>, 128);
    if (need <= 640) return run(w4a16_block_norm_kernel<kX32, 128, 5, 1>, 128);
    if (need <= 768) return run(w4a16_block_norm_kernel<kX32, 128, 6, 1>, 128);
    if (need <= 896) return run(w4a16_block_norm_kernel<kX32, 128, 7, 3>, 128);
    if (need <= 1024) return run(w4a16_block_norm_kernel<kX32, 128, 8, 3>, 128);
  }
  if (need <= 1280) return run(w4a16_block_norm_kernel<kX32, 256, 5, 2>, 256);
  if (need <= 1536) return run(w4a16_block_norm_kernel<kX32, 256, 6, 2>, 256);
  return run(w4a16_block_norm_kernel<kX32, 512, 4, 1>, 512);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& args, int sms, cudaStream_t stream) {
  return args.x_f32 ? launch<true>(args, sms, stream) : launch<false>(args, sms, stream);
}

}  // namespace w4a16
