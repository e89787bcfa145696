// router.cu -- the router's product: logits = x . weight^T, BF16 operands,
// FP32 sums.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace w4a16 {

// One warp per (token, expert).
__global__ void __launch_bounds__(256)
    w4a16_router_logits_kernel(const uint16_t* __restrict__ x, long long x_stride,
                               const uint16_t* __restrict__ weight, int tokens, int hidden,
                               int num_experts, float* __restrict__ logits) {
  const int lane = threadIdx.x & 31;
  const long long total = static_cast<long long>(tokens) * num_experts;
  const long long warps = static_cast<long long>(gridDim.x) * 8;
  for (long long i = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < total;
       i += warps) {
    const long long t = i / num_experts, e = i % num_experts;
    const __nv_bfloat16* xr = reinterpret_cast<const __nv_bfloat16*>(x) + t * x_stride;
    const __nv_bfloat16* wr = reinterpret_cast<const __nv_bfloat16*>(weight) + e * hidden;
    float acc = 0.f;
    for (int c = lane; c < hidden; c += 32)
      acc = fmaf(__bfloat162float(xr[c]), __bfloat162float(wr[c]), acc);
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) logits[i] = acc;
  }
}

cudaError_t launch_router_logits(const uint16_t* x, long long x_stride, const uint16_t* weight,
                                 int tokens, int hidden, int num_experts, float* logits, int sms,
                                 cudaStream_t stream) {
  const long long want = (static_cast<long long>(tokens) * num_experts + 7) / 8;
  const long long cap = static_cast<long long>(sms) * 8;
  w4a16_router_logits_kernel<<<static_cast<int>(want < cap ? want : cap), 256, 0, stream>>>(
      x, x_stride, weight, tokens, hidden, num_experts, logits);
  return cudaGetLastError();
}

}  // namespace w4a16
