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
  // this lane's logits: experts lane, lane + 32, ... (the loads carry no
  // branch, so that all of them are in flight at once); keys order them as
  // integers (0: never chosen; -0 counts as +0; a NaN or a value at or below
  // the lowest finite number is not chosen)
  float v[kPer];
  uint32_t key[kPer];
  float mx = -FLT_MAX;
  const long long row = static_cast<long long>(t) * num_experts;
  if (bf16_logits) {
    const uint16_t* from = static_cast<const uint16_t*>(logits) + row;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      v[i] = __uint_as_float(
          static_cast<uint32_t>(__ldg(from + min(lane + 32 * i, num_experts - 1))) << 16);
  } else {
    const float* from = static_cast<const float*>(logits) + row;
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = __ldg(from + min(lane + 32 * i, num_experts - 1));
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const bool in = lane + 32 * i < num_experts;
    if (!in) v[i] = -FLT_MAX;
    mx = fmaxf(mx, v[i]);
    const uint32_t bits = __float_as_uint(v[i] + 0.f);
    key[i] = v[i] > -FLT_MAX ? ((bits >> 31) != 0 ? ~bits : bits | 0x80000000u) : 0u;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < num_experts) sum += expf(v[i] - mx);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);

  // k rounds of arg-max (largest logit, then lowest id) over the lanes' own
  // best ones, two warp reductions a round. A lane keeps its two largest; it
  // looks through its others only when it has lost both. Lane s keeps round s.
  uint32_t best = 0u, next = 0u, taken = 0u;
  int best_i = 0, next_i = 0;
  const auto two_best = [&]() {
    best = next = 0u;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t k = (taken >> i & 1u) != 0u ? 0u : key[i];
      if (k > best) {
        next = best;
        next_i = best_i;
        best = k;
        best_i = i;
      } else if (k > next) {
        next = k;
        next_i = i;
      }
    }
  };
  two_best();
  float my_v = 0.f;
  int my_id = -1;
#pragma unroll 1
  for (int s = 0; s < topk; ++s) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    if (top == 0u) break;  // no expert left to choose: the other slots hold id -1 and weight 0
    const int e = static_cast<int>(__reduce_min_sync(
        0xffffffffu, best == top ? static_cast<uint32_t>(lane + 32 * best_i) : 0xffffffffu));
    if (lane == s) {
      my_v = __uint_as_float((top >> 31) != 0 ? top & 0x7FFFFFFFu : ~top);
      my_id = e;
    }
    if ((e & 31) == lane) {
      taken |= 1u << best_i;
      best = next;
      best_i = next_i;
      next = 0u;
      if (best == 0u) two_best();
    }
  }
  const float my_p = my_id >= 0 ? expf(my_v - mx) / sum : 0.f;
  float sel_sum = 0.f;
  for (int s = 0; s < topk; ++s) sel_sum += __shfl_sync(0xffffffffu, my_p, s);
  if (lane < topk) {
    const int loc = my_id - expert_offset;
    const long long at = static_cast<long long>(t) * topk + lane;
    topk_ids[at] = (my_id >= 0 && loc >= 0 && loc < num_local) ? loc : -1;
    topk_weights[at] = renormalize ? (sel_sum > 0.f ? my_p / sel_sum : 0.f) : my_p;
  }
}

}  // namespace w4a16
