// route_token.cuh -- top-k routing of one token by one warp, shared by the
// routing kernels (topk.cu) and the few-token layer (moe_few.cu).
#pragma once

#include <cuda_bf16.h>

#include <cfloat>
#include <cstdint>

namespace w4a16 {

// Top-k of token t by one warp (all 32 lanes take part); kPer logits per
// lane, so num_experts <= 32 * kPer.
template <int kPer>
__device__ __forceinline__ void route_token(const void* __restrict__ logits, int bf16_logits, int t,
                                            int num_experts, int topk, int renormalize,
                                            int expert_offset, int num_local,
                                            int32_t* __restrict__ topk_ids,
                                            float* __restrict__ topk_weights) {
  const int lane = threadIdx.x & 31;
  // this lane's logits: experts lane, lane + 32, ...
  float v[kPer];
  float mx = -FLT_MAX;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    v[i] = -FLT_MAX;
    if (e < num_experts) {
      const long long at = static_cast<long long>(t) * num_experts + e;
      v[i] = bf16_logits ? __bfloat162float(static_cast<const __nv_bfloat16*>(logits)[at])
                         : static_cast<const float*>(logits)[at];
      mx = fmaxf(mx, v[i]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < num_experts) sum += expf(v[i] - mx);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);

  // k rounds of arg-max (largest logit, then lowest id); lane s keeps round s
  uint32_t taken = 0;
  float my_p = 0.f, sel_sum = 0.f;
  int my_id = -1;
  for (int s = 0; s < topk; ++s) {
    float bv = -FLT_MAX;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 32 * i;
      if (e < num_experts && !(taken & (1u << i)) && (v[i] > bv || (v[i] == bv && e < be))) {
        bv = v[i];
        be = e;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
      const int oe = __shfl_xor_sync(0xffffffffu, be, o);
      if (ov > bv || (ov == bv && oe < be)) {
        bv = ov;
        be = oe;
      }
    }
    // no expert left to choose (the rest are masked with -inf logits): the
    // slot holds id -1 and weight 0
    const bool found = be < num_experts;
    if (found && (be & 31) == lane) taken |= 1u << (be >> 5);
    const float p = found ? expf(bv - mx) / sum : 0.f;
    sel_sum += p;
    if (lane == s) {
      my_p = p;
      my_id = found ? be : -1;
    }
  }
  if (lane < topk) {
    const int loc = my_id - expert_offset;
    const long long at = static_cast<long long>(t) * topk + lane;
    topk_ids[at] = (my_id >= 0 && loc >= 0 && loc < num_local) ? loc : -1;
    topk_weights[at] = renormalize ? (sel_sum > 0.f ? my_p / sel_sum : 0.f) : my_p;
  }
}

}  // namespace w4a16
