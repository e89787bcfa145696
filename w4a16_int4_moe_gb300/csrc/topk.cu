// topk.cu -- the routing front end: router logits -> top-k local expert ids
// and weights, the inputs of moe_align_block_size.
//
// The pages route every token to the top 8 of 384 experts and hand the
// operator vLLM's routing tensors (page "vLLM 宣布 Humming 后端可运行 … Chord
// 内核 …", section "调度由每个专家收到的 token 数决定"); the router itself is
// the serving stack's. Reading taken here: softmax over all experts, the k
// largest logits (ties to the lower expert id), the chosen probabilities
// optionally renormalised to sum to 1, and global ids mapped to this GPU's
// local experts (-1 for another GPU's). Experts with a -inf logit are masked:
// never chosen; slots that find no expert hold id -1 and weight 0.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "align_cta.cuh"
#include "internal.h"
#include "route_token.cuh"

namespace w4a16 {

namespace {
constexpr int kTopkWarps = 8;       // warps per block, one token per warp
constexpr int kMaxPerLane = 32;     // experts per lane: up to 1024 experts
}  // namespace

template <int kPer>
__global__ void __launch_bounds__(kTopkWarps * 32)
    w4a16_topk_softmax_kernel(const void* __restrict__ logits, int bf16_logits, int tokens,
                              int num_experts, int topk, int renormalize, int expert_offset,
                              int num_local, int32_t* __restrict__ topk_ids,
                              float* __restrict__ topk_weights) {
  const int warps = gridDim.x * kTopkWarps;
  for (int t = blockIdx.x * kTopkWarps + (threadIdx.x >> 5); t < tokens; t += warps)
    route_token<kPer>(logits, bf16_logits, t, num_experts, topk, renormalize, expert_offset,
                      num_local, topk_ids, topk_weights);
}

// Top-k over all CTAs, then moe_align_block_size by the CTA that finishes
// last (it counts the arrivals; no CTA waits on another). `arrivals` is zero
// on entry and reset to zero by that CTA.
template <int kPer>
__global__ void __launch_bounds__(kAlignThreads)
    w4a16_route_align_kernel(const void* __restrict__ logits, int bf16_logits, int tokens,
                             int num_experts, int topk, int renormalize, int expert_offset,
                             int num_local, int block_m, int capacity,
                             int32_t* __restrict__ topk_ids, float* __restrict__ topk_weights,
                             int32_t* __restrict__ sorted_ids, int32_t* __restrict__ expert_ids,
                             int32_t* __restrict__ num_tokens_padded,
                             unsigned int* __restrict__ arrivals) {
  extern __shared__ int smem[];
  __shared__ int is_last;
  // token t goes to CTA t % grid, so that few tokens share an SM
  for (int t = (threadIdx.x >> 5) * gridDim.x + blockIdx.x; t < tokens;
       t += kAlignWarps * gridDim.x)
    route_token<kPer>(logits, bf16_logits, t, num_experts, topk, renormalize, expert_offset,
                      num_local, topk_ids, topk_weights);
  __threadfence();  // this CTA's ids are visible before its arrival counts
  __syncthreads();
  if (threadIdx.x == 0) is_last = atomicAdd(arrivals, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  align_cta(topk_ids, tokens * topk, num_local, block_m, capacity, sorted_ids, expert_ids,
            num_tokens_padded, smem);
  if (threadIdx.x == 0) *arrivals = 0u;
}

namespace {

// pick(logits of a lane): as few as hold the experts, since a warp goes through
// all of them (16384 tokens of 8 experts, top-2: 5.0 us with one, 18 with sixteen;
// 128 experts, top-8: 11 with four, 19 with sixteen). 32 logits a lane, 1024
// experts, stay in the 64 registers that a 1024-thread CTA leaves each thread.
template <typename Pick>
auto by_logits_per_lane(int num_experts, Pick pick) {
  return num_experts <= 32    ? pick(std::integral_constant<int, 1>())
         : num_experts <= 128 ? pick(std::integral_constant<int, 4>())
         : num_experts <= 512 ? pick(std::integral_constant<int, 16>())
                              : pick(std::integral_constant<int, kMaxPerLane>());
}

}  // namespace

cudaError_t launch_topk_softmax(const void* logits, int bf16_logits, int tokens, int num_experts,
                                int topk, int renormalize, int expert_offset, int num_local,
                                int32_t* topk_ids, float* topk_weights, int sms,
                                cudaStream_t stream) {
  if (tokens == 0) return cudaSuccess;
  const int want = (tokens + kTopkWarps - 1) / kTopkWarps;
  const int cap = (sms > 0 ? sms : 1) * 8;
  const auto kernel = by_logits_per_lane(num_experts, [](auto per) {
    return w4a16_topk_softmax_kernel<decltype(per)::value>;
  });
  kernel<<<want < cap ? want : cap, kTopkWarps * 32, 0, stream>>>(
      logits, bf16_logits, tokens, num_experts, topk, renormalize, expert_offset, num_local,
      topk_ids, topk_weights);
  return cudaGetLastError();
}

cudaError_t launch_route_align(const void* logits, int bf16_logits, int tokens, int num_experts,
                               int topk, int renormalize, int expert_offset, int num_local,
                               int block_m, int capacity, int32_t* topk_ids, float* topk_weights,
                               int32_t* sorted_ids, int32_t* expert_ids,
                               int32_t* num_tokens_padded, unsigned int* arrivals, int sms,
                               cudaStream_t stream) {
  const auto kernel = by_logits_per_lane(
      num_experts, [](auto per) { return w4a16_route_align_kernel<decltype(per)::value>; });
  const size_t smem = align_smem_bytes(num_local);
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  // about kTopkWarps tokens per CTA (as the plain top-k launch), up to one
  // CTA per SM
  const int want = (tokens + kTopkWarps - 1) / kTopkWarps;
  const int cap = sms > 0 ? sms : 1;
  const int grid = want < 1 ? 1 : (want < cap ? want : cap);
  kernel<<<grid, kAlignThreads, smem, stream>>>(
      logits, bf16_logits, tokens, num_experts, topk, renormalize, expert_offset, num_local,
      block_m, capacity, topk_ids, topk_weights, sorted_ids, expert_ids, num_tokens_padded,
      arrivals);
  return cudaGetLastError();
}

}  // namespace w4a16
