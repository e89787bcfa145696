// route_token.cuh -- top-k routing of one token by one warp, shared by the
// routing kernels (topk.cu) and the few-token layer (moe_few.cu).
#pragma once

#include <cuda_bf16.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

namespace w4a16 {

// An integer that orders logits as they are ordered: 0 (never chosen) for a NaN
// and for -inf, which masks an expert; the lowest finite value is a logit like
// any other (key 0x00800000), and -0 counts as +0.
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t bits = __float_as_uint(v + 0.f);
  return v >= -FLT_MAX ? ((bits >> 31) != 0 ? ~bits : bits | 0x80000000u) : 0u;
}

// Top-k of token t by one warp (all 32 lanes take part); kPer logits per
// lane, so num_experts <= 32 * kPer.
template <int kPer>
__device__ __forceinline__ void route_token(const void* __restrict__ logits, int bf16_logits, int t,
                                            int num_experts, int topk, int renormalize,
                                            int expert_offset, int num_local,
                                            int32_t* __restrict__ topk_ids,
                                            float* __restrict__ topk_weights) {
  const int lane = threadIdx.x & 31;
  // this lane's logits: experts lane, lane + 32, ... (predicated loads from one
  // address: all of them are in flight at once, and addresses of their own would
  // take more registers than the logits)
  float v[kPer];
  float mx = -FLT_MAX;
  const long long first = static_cast<long long>(t) * num_experts + lane;
  const int mine = num_experts - lane;
  if (bf16_logits) {
    const uint16_t* from = static_cast<const uint16_t*>(logits) + first;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      v[i] = 32 * i < mine ? __uint_as_float(static_cast<uint32_t>(__ldg(from + 32 * i)) << 16)
                           : -INFINITY;
  } else {
    const float* from = static_cast<const float*>(logits) + first;
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = 32 * i < mine ? __ldg(from + 32 * i) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) mx = fmaxf(mx, v[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < num_experts) sum += expf(v[i] - mx);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);

  uint32_t key[kPer];  // (from here on in place of the logits)
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = logit_key(v[i]);
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

// The same by a whole CTA of kWarps warps (all threads take part), for one
// token at a time: the shortest way through when there are few. Warp w takes
// the experts of the rows 32 i .. 32 i + 31, i = w, w + kWarps, ..., and sorts
// out its topk best; warp 0 merges the lists. Results, to the bit, as above
// (the exponentials are added in the same order). scratch: 32 * 32 + 2 *
// kWarps * 32 + kWarps words of shared memory; ids and weights may be shared
// memory too.
template <int kWarps>
__device__ __forceinline__ void route_token_cta(const void* __restrict__ logits, int bf16_logits,
                                                int t, int num_experts, int topk, int renormalize,
                                                int expert_offset, int num_local, int32_t* ids,
                                                float* weights, float* scratch) {
  constexpr int kRows = (32 + kWarps - 1) / kWarps;
  float* exps = scratch;  // [32][32]
  uint32_t* list_key = reinterpret_cast<uint32_t*>(scratch + 32 * 32);  // [kWarps][32]
  int* list_id = reinterpret_cast<int*>(list_key + kWarps * 32);
  float* tops = reinterpret_cast<float*>(list_id + kWarps * 32);  // [kWarps]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = (num_experts + 31) / 32;
  const long long row = static_cast<long long>(t) * num_experts;
  float v[kRows];
  uint32_t key[kRows];
  float mx = -FLT_MAX;
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int e = min(32 * (warp + j * kWarps) + lane, num_experts - 1);
    v[j] = bf16_logits ? __uint_as_float(static_cast<uint32_t>(
                                             __ldg(static_cast<const uint16_t*>(logits) + row + e))
                                         << 16)
                       : __ldg(static_cast<const float*>(logits) + row + e);
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    if (32 * (warp + j * kWarps) + lane >= num_experts) v[j] = -INFINITY;
    mx = fmaxf(mx, v[j]);
    key[j] = logit_key(v[j]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) tops[warp] = mx;
  // this warp's topk best, largest first, ties to the lower expert
  uint32_t my_key = 0u;
  int my_id = -1;
#pragma unroll 1
  for (int s = 0; s < topk; ++s) {
    uint32_t best = 0u;
    int best_j = 0;
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      if (key[j] > best) {
        best = key[j];
        best_j = j;
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    if (top == 0u) break;
    const int e = static_cast<int>(__reduce_min_sync(
        0xffffffffu,
        best == top ? static_cast<uint32_t>(32 * (warp + best_j * kWarps) + lane) : 0xffffffffu));
    if ((e & 31) == lane && best == top)
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        if (j == best_j) key[j] = 0u;
    if (lane == s) {
      my_key = top;
      my_id = e;
    }
  }
  list_key[warp * 32 + lane] = my_key;
  list_id[warp * 32 + lane] = my_id;
  __syncthreads();
  mx = -FLT_MAX;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, tops[w]);
#pragma unroll
  for (int j = 0; j < kRows; ++j)
    if (warp + j * kWarps < rows)
      exps[(warp + j * kWarps) * 32 + lane] =
          32 * (warp + j * kWarps) + lane < num_experts ? expf(v[j] - mx) : 0.f;
  __syncthreads();
  if (warp == 0) {
    float sum = 0.f;
    for (int i = 0; i < rows; ++i) sum += exps[i * 32 + lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // lane w walks list w
    int pos = 0;
    uint32_t head = lane < kWarps ? list_key[lane * 32] : 0u;
    int head_id = lane < kWarps ? list_id[lane * 32] : -1;
    float my_v = 0.f;
    my_id = -1;
#pragma unroll 1
    for (int s = 0; s < topk; ++s) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, head);
      if (top == 0u) break;
      const int e = static_cast<int>(__reduce_min_sync(
          0xffffffffu, head == top ? static_cast<uint32_t>(head_id) : 0xffffffffu));
      if (lane == s) {
        my_v = __uint_as_float((top >> 31) != 0 ? top & 0x7FFFFFFFu : ~top);
        my_id = e;
      }
      if (head == top && head_id == e) {
        ++pos;
        head = pos < topk ? list_key[lane * 32 + pos] : 0u;
        head_id = pos < topk ? list_id[lane * 32 + pos] : -1;
      }
    }
    const float my_p = my_id >= 0 ? expf(my_v - mx) / sum : 0.f;
    float sel_sum = 0.f;
    for (int s = 0; s < topk; ++s) sel_sum += __shfl_sync(0xffffffffu, my_p, s);
    if (lane < topk) {
      const int loc = my_id - expert_offset;
      const long long at = static_cast<long long>(t) * topk + lane;
      ids[at] = (my_id >= 0 && loc >= 0 && loc < num_local) ? loc : -1;
      weights[at] = renormalize ? (sel_sum > 0.f ? my_p / sel_sum : 0.f) : my_p;
    }
  }
  __syncthreads();  // scratch is free again
}

}  // namespace w4a16
