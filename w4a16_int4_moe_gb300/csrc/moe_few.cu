// moe_few.cu -- a whole MoE layer for a few tokens: routing, gate_up, the
// activation, down and the top-k weighted sum.
//
// Weights (q - 8) * scale, the activation and every sum are kept in FP32.

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace w4a16 {

namespace {

__device__ __forceinline__ float bf16_value(uint16_t bits) {
  return __uint_as_float(static_cast<uint32_t>(bits) << 16);
}

__device__ __forceinline__ float e4m3_value(uint8_t bits) {
  return __half2float(__nv_cvt_fp8_to_halfraw(bits, __NV_E4M3));
}

// sum over the lane's groups of 32 columns of row `row` of packed tile
// `tile`, times value(column)
template <typename Value>
__device__ float packed_dot(const uint8_t* expert, int k, int tile, int row, Value value) {
  const int lane = threadIdx.x & 31;
  const int k_steps = (k + kKStep - 1) / kKStep;
  float acc = 0.f;
  for (int g = lane; g < k / kGroup; g += 32) {
    const uint8_t* step =
        expert + (static_cast<long long>(tile) * k_steps + g / 2) * static_cast<long long>(kStepBytes);
    const uint4 q = *reinterpret_cast<const uint4*>(step + (g & 1) * (kTileRows * 16) + row * 16);
    const float scale = bf16_value(*reinterpret_cast<const uint16_t*>(
        step + kStepQBytes + (g & 1) * (kTileRows * 2) + row * 2));
    const uint32_t words[4] = {q.x, q.y, q.z, q.w};
    float sum = 0.f;
    for (int j = 0; j < 4; ++j)
      for (int i = 0; i < 4; ++i) {  // word j, bits 4i: k = 8j + 2i, bits 16 + 4i: k + 1
        const int c = g * kGroup + 8 * j + 2 * i;
        const int lo = static_cast<int>((words[j] >> (4 * i)) & 15u) - 8;
        const int hi = static_cast<int>((words[j] >> (16 + 4 * i)) & 15u) - 8;
        sum = fmaf(static_cast<float>(lo), value(c), sum);
        sum = fmaf(static_cast<float>(hi), value(c + 1), sum);
      }
    acc = fmaf(scale, sum, acc);
  }
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  return acc;
}

}  // namespace

// One warp per (pick, activation column).
__global__ void __launch_bounds__(256) w4a16_few_gate_up_kernel(const FewArgs a, float* act) {
  const int groups = (a.hidden + 127) / 128;
  const long long total = static_cast<long long>(a.tokens) * a.topk * a.inter;
  for (long long i = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < total;
       i += static_cast<long long>(gridDim.x) * 8) {
    const int pick = static_cast<int>(i / a.inter), c = static_cast<int>(i % a.inter);
    const int e = a.topk_ids[pick];
    if (e < 0 || e >= a.num_experts) continue;
    const long long t = pick / a.topk;
    auto value = [&](int k) {
      if (!a.x_fp8) return bf16_value(static_cast<const uint16_t*>(a.x)[t * a.hidden + k]);
      return e4m3_value(static_cast<const uint8_t*>(a.x)[t * a.hidden + k]) *
             a.x_scales[t * groups + k / 128];
    };
    // gate row c and up row inter + c of the interleaved packing
    const uint8_t* expert = a.gate_up + e * a.gate_up_expert_bytes;
    const int row = (c % 64) / 16 * 32 + c % 16;
    const float g = packed_dot(expert, a.hidden, c / 64, row, value);
    const float u = packed_dot(expert, a.hidden, c / 64, row + 16, value);
    if ((threadIdx.x & 31) == 0) act[i] = g / (1.f + expf(-g)) * u;
  }
}

// One warp per output element.
__global__ void __launch_bounds__(256) w4a16_few_down_kernel(const FewArgs a, const float* act) {
  const long long total = static_cast<long long>(a.tokens) * a.hidden;
  for (long long i = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < total;
       i += static_cast<long long>(gridDim.x) * 8) {
    const int t = static_cast<int>(i / a.hidden), c = static_cast<int>(i % a.hidden);
    float sum = 0.f;
    for (int s = 0; s < a.topk; ++s) {
      const int pick = t * a.topk + s;
      const int e = a.topk_ids[pick];
      if (e < 0 || e >= a.num_experts) continue;
      const float* row = act + static_cast<long long>(pick) * a.inter;
      const float d = packed_dot(a.down + e * a.down_expert_bytes, a.inter, c / kTileRows,
                                 c % kTileRows, [&](int k) { return row[k]; });
      sum = fmaf(a.topk_weights[pick], d, sum);
    }
    if ((threadIdx.x & 31) == 0) a.out[i] = a.accumulate ? a.out[i] + sum : sum;
  }
}

size_t few_workspace_bytes(int tokens, int topk, int hidden, int inter) {
  (void)hidden;
  return kStatusBytes + static_cast<size_t>(tokens) * topk * inter * sizeof(float);
}

cudaError_t launch_moe_few(const FewArgs& args, int sms, cudaStream_t stream) {
  if (args.logits != nullptr) {
    const cudaError_t e = launch_topk_softmax(
        args.logits, args.bf16_logits, args.tokens, args.num_global, args.topk, args.renormalize,
        args.expert_offset, args.num_experts, args.topk_ids, args.topk_weights, sms, stream);
    if (e != cudaSuccess) return e;
  }
  float* act = reinterpret_cast<float*>(args.workspace + kStatusBytes);
  w4a16_few_gate_up_kernel<<<sms * 8, 256, 0, stream>>>(args, act);
  w4a16_few_down_kernel<<<sms * 8, 256, 0, stream>>>(args, act);
  return cudaGetLastError();
}

}  // namespace w4a16
