// products.cu -- products with one weight, BF16 or packed INT4, plain or gated:
//
//   out[t, r] = addend[t, r] + x[t] . w[r]^T
//   out[t, i] = silu(x[t] . wgate[i]^T) * (x[t] . wup[i]^T)
//
// The simplest form that is right for every case: a CTA has 16 tokens and 16
// columns of the output, a thread one value, and both operands come through
// shared memory 32 columns at a time in FP32.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace w4a16 {

namespace {

constexpr int kEdge = 16;

__device__ __forceinline__ float from_bf16(uint16_t v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// Weight (row of the packed tiles, column c).
__device__ __forceinline__ float packed_value(const uint8_t* packed, int k, int row, int c) {
  const int steps = (k + kKStep - 1) / kKStep;
  const uint8_t* step =
      packed + (static_cast<long long>(row / kTileRows) * steps + c / kKStep) * kStepBytes;
  const int r = row % kTileRows, g = c / kGroup % 2, j = c % kGroup;
  const uint32_t word =
      *reinterpret_cast<const uint32_t*>(step + g * (kTileRows * 16) + r * 16 + j / 8 * 4);
  const int code = static_cast<int>(word >> (j % 8 / 2 * 4 + j % 2 * 16) & 15u);
  const uint16_t scale =
      *reinterpret_cast<const uint16_t*>(step + kStepQBytes + g * (kTileRows * 2) + r * 2);
  return static_cast<float>(code - 8) * from_bf16(scale);
}

}  // namespace

template <bool kInt4>
__global__ void __launch_bounds__(kEdge * kEdge) w4a16_product_kernel(const ProductArgs a) {
  __shared__ float xs[kEdge][kGroup + 1], ws[2][kEdge][kGroup + 1];
  const int tx = threadIdx.x % kEdge, ty = threadIdx.x / kEdge;
  const int columns = a.gated ? a.n / 2 : a.n;
  const int r0 = blockIdx.x * kEdge;
  grid_dependency_wait();
  grid_dependents_go();
  for (int t0 = blockIdx.y * kEdge; t0 < a.tokens; t0 += gridDim.y * kEdge) {
    float sum[2] = {};
    for (int k0 = 0; k0 < a.k; k0 += kGroup) {
      __syncthreads();
      for (int i = threadIdx.x; i < kEdge * kGroup; i += kEdge * kEdge) {
        const int row = i / kGroup, c = k0 + i % kGroup;
        const bool in = c < a.k && t0 + row < a.tokens;
        xs[row][i % kGroup] = in ? from_bf16(a.x[(t0 + row) * a.x_stride + c]) : 0.f;
        const int r = r0 + row;
        for (int half = 0; half <= a.gated; ++half) {
          float v = 0.f;
          if (r < columns && c < a.k) {
            if constexpr (kInt4) {
              const int p = a.gated ? r / 64 * 128 + r % 64 / 16 * 32 + r % 16 + half * 16 : r;
              v = packed_value(static_cast<const uint8_t*>(a.weight), a.k, p, c);
            } else {
              v = from_bf16(static_cast<const uint16_t*>(
                  a.weight)[static_cast<long long>(half * columns + r) * a.k + c]);
            }
          }
          ws[half][row][i % kGroup] = v;
        }
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kGroup; ++c) {
        sum[0] = fmaf(xs[ty][c], ws[0][tx][c], sum[0]);
        if (a.gated) sum[1] = fmaf(xs[ty][c], ws[1][tx][c], sum[1]);
      }
    }
    const int t = t0 + ty, r = r0 + tx;
    if (t >= a.tokens || r >= columns) continue;
    const long long at = static_cast<long long>(t) * columns + r;
    float v = a.gated ? sum[0] / (1.f + expf(-sum[0])) * sum[1] : sum[0];
    if (a.addend != nullptr) v += a.addend[at];
    if (a.f32_out)
      static_cast<float*>(a.out)[at] = v;
    else
      static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
  }
}

namespace {

template <bool kInt4>
cudaError_t launch_product(const ProductArgs& a, cudaStream_t stream) {
  const int columns = a.gated ? a.n / 2 : a.n;
  const dim3 grid(static_cast<unsigned>(ceil_div(columns, kEdge)),
                  static_cast<unsigned>(std::min(ceil_div(a.tokens, kEdge), 32768)));
  w4a16_product_kernel<kInt4><<<grid, kEdge * kEdge, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dense(const ProductArgs& args, int sms, cudaStream_t stream) {
  if (args.tokens <= kDenseFewTokens) return launch_dense_few(args, sms, stream);
  return launch_product<false>(args, stream);
}

}  // namespace w4a16
