// product_tmem.cu -- products with one packed INT4 weight of many rows for 17 to 32
// tokens, plain or gated:
//
//   out[t, r] = addend[t, r] + x[t] . w[r]^T
//   out[t, i] = silu(x[t] . wgate[i]^T) * (x[t] . wup[i]^T)
//
// 128 weight rows are the M side of tcgen05 MMAs and the tokens their N side. The
// codes become BF16 numbers q - 8 in TMEM; each group of 32 columns has sums of its
// own there, which times the group's scale are added up in FP32 registers, so no
// weight is rounded.
//
// 32 tokens of 16384 x 7168 in a graph: 23.5 us, 2.8 TB/s of the weight; with
// mma.sync, whose accumulators go through the same FP32 additions, 32.8: beside
// them a scheduler starts an MMA in 12.8 cycles instead of 8.5. Here a step takes a
// scheduler 330 cycles, in which it issues 220 instructions, 96 of them for the
// conversion and 32 for the additions; without the conversion it takes 50 cycles
// less, with a quarter of the MMAs 20, without the additions 40. Warps of one kind
// each, which hand steps to one another through barriers, took 28.7 us, a ring of
// two units for three 25.4.

#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "pipe.cuh"
#include "product_out.cuh"
#include "ptx.cuh"

namespace w4a16 {

namespace {

constexpr int kTokens = 32;         // the N side
constexpr int kGroups = 4;          // warpgroups
constexpr int kGroupThreads = 128;  // a weight row, and a TMEM lane, each
constexpr int kTmemThreads = kGroups * kGroupThreads;
constexpr int kUnit = 2;            // steps of a slot of the ring, each with a buffer in TMEM
constexpr int kRing = 3;            // slots of a group
// Barriers of a group: slots that are full, MMAs that are done, and for each issuing
// warp that its last MMAs are over.
constexpr int kBars = kRing + 1 + kUnit;
constexpr int kPitch = kTileRows + kSumPad;  // of a token's sums
// A group's columns of TMEM: the sums of a step's two halves, then the buffers.
constexpr int kGroupColumns = 512 / kGroups, kNumbersAt = 2 * kTokens, kNumbers = kKStep / 2;
static_assert(kNumbersAt + kUnit * kNumbers <= kGroupColumns, "TMEM");
// A slot: the tokens' columns of each step, then the codes and scales.
constexpr uint32_t kXBytes = kTokens * kKStep * 2, kCodes = kUnit * kXBytes;
constexpr uint32_t kUnitBytes = kCodes + kUnit * kStepBytes;
static_assert(kUnitBytes % 1024 == 0, "swizzled tiles");
constexpr int kTmemSmem = 1024 + kGroups * kRing * kUnitBytes + kTokens * kPitch * 4;
static_assert(kTmemSmem <= kMaxSmem, "shared memory of an SM");

struct TmemProduct {
  CUtensorMap x;
  ProductArgs a;
  int blocks;         // of 128 weight rows
  int steps;          // of 64 columns
  uint32_t sixteens;  // 16 as two BF16 numbers
  long long wait_limit;  // cycles
};

// The warps of a group meet where one of them goes on for all, at two barriers by
// turns. None comes to a barrier again before all have left it: one that arrives and
// goes on waits next for the MMAs that are issued behind the barrier, and one of which
// a wait gave up, and which waits for nothing else any more, stays at every barrier
// until all are there. (Else its arrivals would stand in for those of others, and who
// stays would stay for ever.)
__device__ __forceinline__ void group_wait(int barrier) {
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "n"(kGroupThreads) : "memory");
}
__device__ __forceinline__ void group_arrive(int barrier) {
  asm volatile("bar.arrive %0, %1;" ::"r"(barrier), "n"(kGroupThreads) : "memory");
}

}  // namespace

// Four warpgroups take units of two steps by turns, each for itself and from a
// ring of its own, which it fills again itself: x by TMA, the codes and scales,
// which lie together, by a bulk copy. It converts a step into TMEM while the tensor
// core has the one before, adds that one's sums and issues this one's MMAs.
template <bool kGated>
__global__ void __launch_bounds__(kTmemThreads, 1)
    w4a16_product_tmem_kernel(const __grid_constant__ TmemProduct p) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* part = reinterpret_cast<float*>(smem + kGroups * kRing * kUnitBytes);  // [kTokens][kPitch]
  __shared__ uint64_t bars[kGroups * kBars];
  __shared__ uint32_t tmem_at;
  __shared__ int failed_word;
  volatile int* failed = &failed_word;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const int group = warp / 4, row = warp % 4 * 32 + lane;
  const uint32_t full = smem_u32(bars + group * kBars), done = full + 8 * kRing,
                 idle = done + 8;
  const uint32_t ring = smem_u32(smem) + group * (kRing * kUnitBytes);
  const int begin = static_cast<int>(blockIdx.x), stride = static_cast<int>(gridDim.x);
  const int units = (p.steps + kUnit - 1) / kUnit;
  // The first weights set out while the kernel before is at work (0.3 us less).
  if (warp % 4 == 1 && elect_one())
    for (int i = 0; i < kRing && group + i * kGroups < units; ++i) {
      const int step = (group + i * kGroups) * kUnit;
      prefetch_l2_range(static_cast<const uint8_t*>(p.a.weight) +
                            (static_cast<long long>(begin) * p.steps + step) * kStepBytes,
                        min(kUnit, p.steps - step) * kStepBytes);
    }
  __syncwarp();
  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < kGroups * kBars; ++i) mbar_init(smem_u32(bars + i), 1);
      *failed = 0;
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(smem_u32(&tmem_at), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();
  grid_dependents_go();
  const uint32_t tmem = tmem_at;
  const uint32_t idesc = idesc_bf16_m128(kTokens);
  const uint32_t columns = tmem + group * kGroupColumns;
  const uint32_t lanes = columns + (static_cast<uint32_t>(warp % 4 * 32) << 16);
  const uint64_t once = policy_evict_first();
  // The group's next unit to copy: one by one it takes every fourth of a block's,
  // then goes on in the next block.
  int next_block = begin, next_unit = group, fetched = 0;
  Ring to;
  const auto fetch = [&] {  // (warp 0 of the group)
    while (next_unit >= units && next_block < p.blocks) {
      next_unit = group;
      next_block = units > group ? next_block + stride : p.blocks;
    }
    if (next_block >= p.blocks) return;
    if (elect_one()) {
      const int step = next_unit * kUnit, n = min(kUnit, p.steps - step);
      const uint32_t at = ring + to.slot * kUnitBytes, bar = full + 8 * to.slot;
      mbar_arrive_expect_tx(bar, n * (kXBytes + kStepBytes));
      bulk_g2s(at + kCodes,
               static_cast<const uint8_t*>(p.a.weight) +
                   (static_cast<long long>(next_block) * p.steps + step) * kStepBytes,
               n * kStepBytes, bar, once);
      for (int j = 0; j < n; ++j)
        tma_load_2d(at + j * kXBytes, &p.x, (step + j) * kKStep, 0, bar);
    }
    __syncwarp();
    ++fetched;
    next_unit += kGroups;
    to.next(kRing);
  };
  if (warp % 4 == 0)
    for (int i = 0; i < kRing; ++i) fetch();
  Ring r;
  uint32_t phase = 0;
  bool ok = true;  // no wait of this warp has given up
  float sum[kTokens];
  // A step's codes into buffer j.
  const auto convert = [&](const uint4 (&codes)[2], int j) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t q[4] = {codes[h].x, codes[h].y, codes[h].z, codes[h].w};
      uint32_t v[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[4 * i] = code_pair(q[i] << 3, p.sixteens);
        v[4 * i + 1] = code_pair(q[i] >> 1, p.sixteens);
        v[4 * i + 2] = code_pair(q[i] >> 5, p.sixteens);
        v[4 * i + 3] = code_pair(q[i] >> 9, p.sixteens);
      }
      tmem_st_32x32b_x16(lanes + kNumbersAt + j * kNumbers + h * 16, v);
    }
  };
  // The sums of the step whose scales lie at `scales`, once its MMAs are done: 16
  // columns at a time, while the next ones are on their way. False if they never are.
  const auto add = [&](uint32_t scales) {
    const bool there = ring_wait<false>(done, phase, failed, p.wait_limit);
    if (!__all_sync(0xffffffffu, there)) return false;
    phase ^= 1u;
    tc_fence_after();
    uint32_t v[2][16];
    tmem_ld_32x32b_x16(lanes, v[0]);
    const float scale[2] = {load_scale(scales), load_scale(scales + kTileRows * 2)};
#pragma unroll
    for (int i = 0; i < kTokens / 8; ++i) {
      tmem_ld_wait_for(v[i % 2]);
      if (i + 1 < kTokens / 8) tmem_ld_32x32b_x16(lanes + (i + 1) * 16, v[(i + 1) % 2]);
      const int t0 = i * 16 % kTokens;
#pragma unroll
      for (int c = 0; c < 16; c += 2)
        fma_pair(sum[t0 + c], sum[t0 + c + 1], scale[i * 16 / kTokens],
                 __uint_as_float(v[i % 2][c]), __uint_as_float(v[i % 2][c + 1]));
    }
    return true;
  };
  // The MMAs of buffer j, by one warp (another one for each j) once all four have
  // converted their rows and read the sums of before; the others go on. Then the
  // slot of the unit before is free.
  int barrier = 2 + 2 * group;  // and the next one (0 is that of the whole CTA)
  const auto multiply = [&](uint32_t x_at, int j, bool refill) {
    tmem_st_wait();
    tc_fence_before();
    const int here = barrier;
    barrier ^= 1;
    if (warp % 4 != j) {
      group_arrive(here);
      return;
    }
    group_wait(here);
    tc_fence_after();
    if (elect_one()) {
      const uint64_t x = smem_desc_sw128_kmajor(x_at);
#pragma unroll
      for (int i = 0; i < 4; ++i)  // 16 columns: 8 of TMEM, 32 bytes of x
        mma_bf16_ts(columns + i / 2 * kTokens, columns + kNumbersAt + j * kNumbers + i * 8,
                    x + 2 * i, idesc, i & 1);
      tc_commit(done);
    }
    __syncwarp();
    if (j == 0 && refill) fetch();
  };
  const uint32_t codes_at = kCodes + row * 16, scales_at = kCodes + kStepQBytes + row * 2;
  // the group's steps of a block
  const int steps = units <= group ? 0 : (units - 1 - group) / kGroups * kUnit + kUnit -
                                             ((units - 1 - group) % kGroups == 0 && p.steps % kUnit);
  for (int block = begin; block < p.blocks; block += stride) {
#pragma unroll
    for (int i = 0; i < kTokens; ++i) sum[i] = 0.f;
    uint32_t under = 0;  // scales of the step under way
    int left = ok ? 0 : steps;  // that this warp takes no part in
    for (int unit = ok ? group : units; unit < units; unit += kGroups, r.next(kRing)) {
      const auto give_up_at = [&](int j) {  // with step j of this unit
        ok = false;
        left = steps - (unit - group) / kGroups * kUnit - j;
      };
      const uint32_t slot = ring + r.slot * kUnitBytes;
      const bool there = ring_wait<false, true>(full + 8 * r.slot, r.phase, failed, p.wait_limit);
      if (!__all_sync(0xffffffffu, there)) {
        give_up_at(0);
        break;
      }
      uint4 w[kUnit][2];
#pragma unroll
      for (int j = 0; j < kUnit; ++j)  // (behind the last step: not used)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[j][h] = load_shared16(slot + codes_at + j * kStepBytes + h * (kTileRows * 16));
      convert(w[0], 0);
      if (under != 0 && !add(under)) {
        give_up_at(0);
        break;
      }
      multiply(slot, 0, under != 0);
      under = slot + scales_at;
      if (unit * kUnit + 1 < p.steps) {
        convert(w[1], 1);
        if (!add(under)) {
          give_up_at(1);
          break;
        }
        multiply(slot + kXBytes, 1, false);
        under += kStepBytes;
      }
    }
    if (ok && under != 0) ok = add(under);
    for (tmem_st_wait(); left > 0; --left, barrier ^= 1) group_wait(barrier);
    // the sums of one group on to those of the others
    const float nan = __uint_as_float(0x7FC00000u);
    float* mine = part + row;
    __syncthreads();  // the block before is out, and the last unit's slot free
    if (warp % 4 == 0 && under != 0 && ok) fetch();
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (group == g)
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
          const float before = g > 0 ? mine[i * kPitch] : 0.f;
          mine[i * kPitch] = ok ? before + sum[i] : nan;
        }
      if (g + 1 < kGroups) __syncthreads();
    }
    __syncthreads();
    write_products<kGated, kTileRows>(p.a, part, block, static_cast<int>(threadIdx.x),
                                      kTmemThreads, 1);
  }
  // Copies and MMAs in flight are over before the CTA ends. (Where no wait gave up all
  // were waited for, and from then on no more are copied.)
  if (!ok && warp % 4 == 0)
    for (int i = max(0, fetched - kRing); i < fetched; ++i)
      drain<false>(full + 8 * (i % kRing), i / kRing & 1);
  if (!ok && warp % 4 < kUnit && elect_one()) {
    tc_commit(idle + 8 * (warp % 4));  // of this thread's MMAs
    drain<false>(idle + 8 * (warp % 4), 0);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

cudaError_t launch_linear_tmem(const ProductArgs& args, int sms, cudaStream_t stream) {
  const auto kernel =
      args.gated ? w4a16_product_tmem_kernel<true> : w4a16_product_tmem_kernel<false>;
  TmemProduct p;
  if (!encode_rows_tmap(&p.x, args.x, args.tokens, args.k, args.x_stride, kTokens))
    return cudaErrorInvalidValue;
  p.a = args;
  p.sixteens = 0x41804180u;
  p.wait_limit = wait_timeout_cycles();
  p.blocks = ceil_div(args.n, kTileRows);
  p.steps = ceil_div(args.k, kKStep);
  static Devices known[2];
  const cudaError_t e = allow_smem(kernel, kTmemSmem, known[args.gated ? 1 : 0]);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, std::min(p.blocks, sms), kTmemThreads, kTmemSmem, 1, stream, p);
}

}  // namespace w4a16
