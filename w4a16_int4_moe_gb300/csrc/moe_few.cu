// moe_few.cu -- a whole MoE layer for a few tokens in one launch: routing,
// gate_up, the activation, down and the top-k weighted sum.
//
//   act[r]  = silu(x[t] . Wgate_e^T) * (x[t] . Wup_e^T)     for each row r = (e, t)
//   out[t]  = sum over the rows r of t of weight[r] * (act[r] . Wdown_e^T)
//
// A few tokens use every weight of a chosen expert for one to a few rows, so
// the packed weights are the whole traffic and the layer is bound by reading
// them once. The kernel is built around that stream:
//
//   * one persistent CTA per SM; both products are cut into stages of 128
//     weight rows x 128 k (9216 packed bytes) and every CTA takes an equal,
//     contiguous run of them, first of gate_up, then of down, so that all SMs
//     read the same number of bytes whatever the number of experts;
//   * two threads copy the stages into a shared-memory ring (bulk copies);
//     they run through both products without waiting for the activation, so
//     the ring is full of down weights when the activation is complete;
//   * sixteen warps turn the codes into 16-bit integers in registers and feed
//     them to m16n8k16 MMAs: weights are the M side, the rows of an expert
//     (at most eight per pass over its weights) the N side. q - 8 is exact in
//     16 bits; the scale of a group of 32 is applied to the group's FP32 sum,
//     so no weight is rounded. The dequantised weights never leave registers:
//     through TMEM, as the tcgen05 kernel of the large batches needs them, the
//     same stream reaches 0.4 of the copy bandwidth;
//   * the activation is handed to the second product as three BF16 parts whose
//     sum is the FP32 value (each part cuts off 8 bits): one or two rows put
//     their parts into different columns of one MMA, more rows take three
//     MMAs into one accumulator;
//   * two warps finish the items from shared memory while the others go on.
//
// An item (gate_up: one tile of one expert; down: one tile over all experts)
// may be cut between CTAs: each writes its FP32 share to the workspace and
// the CTA that arrives last adds the shares in order. Nothing is added with
// atomics, so the result depends only on the sizes and the routing.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"
#include "route_token.cuh"

namespace w4a16 {

namespace {

constexpr int kGroups = 4;                   // warpgroups; group g takes every fourth stage
constexpr int kComputeWarps = 4 * kGroups;
constexpr int kComputeThreads = 32 * kComputeWarps;
// Two warps issue the weight copies by turns: one thread gets round its loop
// (wait for the slot, announce the bytes, copy) only every 620 cycles, 4.4 TB/s
// of 9216-byte stages on 152 SMs; two reach 7.1 TB/s.
constexpr int kWeightWarps = 2;
constexpr int kWarpWeights0 = kComputeWarps;
constexpr int kWarpEpilogue0 = kComputeWarps + kWeightWarps;
constexpr int kEpilogueWarps = 2;
constexpr int kEpilogueThreads = 32 * kEpilogueWarps;
constexpr int kFewThreads = kComputeThreads + 32 * kWeightWarps + kEpilogueThreads;
constexpr int kWStage = 2 * kStepBytes;      // packed bytes of a stage: two 64-k steps
constexpr int kStageK = 2 * kKStep;
constexpr int kRowsPerPass = 8;              // rows of an expert per pass over its weights (MMA N)
constexpr int kParts = 3;                    // BF16 parts of an activation value
constexpr int kSumPitch = 132;               // FP32 sums [row][128 + 4]
constexpr int kMaxCtas = 192;
constexpr int kMinSlots = 4;
constexpr int kMaxSlots = 16;  // 147 KB in flight (more measured slower)
constexpr int kFewMaxSmem = 232448;
constexpr long long kFewDrainCycles = 4000000000LL;

// waits that can give up (status word detail)
enum { kWhereRing = 0x21, kWhereData = 0x22, kWhereAct = 0x23, kWhereSums = 0x24 };

// Workspace: status words, counters, the CTAs' shares, the activation parts.
struct FewCounters {
  int act_done;               // finished gate_up items
  int exits;                  // CTAs that are through
  int pad[2];
  int item[2][kMaxCtas];      // arrivals at the item that a CTA begins and does not finish
};
constexpr size_t kCounterBytes = (sizeof(FewCounters) + 255) / 256 * 256;

__host__ __device__ inline int max_rows(int tokens, int topk) { return tokens * topk; }
__host__ __device__ inline size_t share_floats(int tokens) {
  return static_cast<size_t>(tokens > kRowsPerPass ? tokens : kRowsPerPass) * kTileRows;
}

// FP32 sums: two buffers of an item's sums by warpgroup (gate_up), or one of
// a tile's by warpgroup (down).
constexpr int kItemSums = kGroups * kRowsPerPass * kSumPitch;
inline int sum_floats(int tokens) { return std::max(2 * kItemSums, kGroups * tokens * kSumPitch); }

// Shared memory of a call, all offsets in bytes.
struct FewSmem {
  int slots, ring;
  int sums, ids, weights, mask, base, row_token, row_weight, chunks, x_scales, total;
};
FewSmem few_smem(int tokens, int topk, int num_experts, int hidden, bool fp8) {
  FewSmem s;
  const int rows = max_rows(tokens, topk);
  int at = 1024;  // barriers and scalars
  auto take = [&at](size_t bytes) {
    const int here = at;
    at += static_cast<int>((bytes + 127) / 128 * 128);
    return here;
  };
  s.sums = take(sizeof(float) * sum_floats(tokens));
  s.ids = take(4 * static_cast<size_t>(rows));
  s.weights = take(4 * static_cast<size_t>(rows));
  s.mask = take(4 * static_cast<size_t>(num_experts));
  s.base = take(4 * static_cast<size_t>(num_experts));
  s.row_token = take(4 * static_cast<size_t>(rows));
  s.row_weight = take(4 * static_cast<size_t>(rows));
  s.chunks = take(4 * static_cast<size_t>(rows));
  s.x_scales = take(fp8 ? 4 * static_cast<size_t>(tokens) * ((hidden + 127) / 128) : 0);
  s.ring = at;
  s.slots = std::min(kMaxSlots, (kFewMaxSmem - at) / kWStage);
  s.total = at + s.slots * kWStage;
  return s;
}

struct FewParams {
  FewArgs a;
  FewSmem s;
};

// ------------------------------------------------------------------ MMA ---

// c = a . b (first) or c + a . b
template <bool kF16, bool kFirst>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  const float i0 = kFirst ? 0.f : c[0], i1 = kFirst ? 0.f : c[1], i2 = kFirst ? 0.f : c[2],
              i3 = kFirst ? 0.f : c[3];
  if constexpr (kF16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(i0), "f"(i1),
          "f"(i2), "f"(i3));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(i0), "f"(i1),
          "f"(i2), "f"(i3));
  }
}

// (volatile keeps them behind the wait for their slot and before its release)
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr));
}

// Codes 2i and 2i + 1 of a packed word as the pair (q - 8, q - 8): the nibble
// becomes the low mantissa bits of 128 (BF16) or 1024 (FP16), the difference
// to 136 or 1032 is exact.
template <bool kF16>
__device__ __forceinline__ uint32_t code_pair(uint32_t word, int i) {
  constexpr uint32_t kBase = kF16 ? 0x64006400u : 0x43004300u;
  constexpr uint32_t kZero = kF16 ? 0x64086408u : 0x43084308u;
  const uint32_t v = ((word >> (4 * i)) & 0x000F000Fu) | kBase;
  uint32_t r;
  if constexpr (kF16)
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(kZero));
  else
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(kZero));
  return r;
}

__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(r)
      : "r"(two));
  return r;
}

// The column values of a lane, two groups of 32 k: thread t of a quad takes
// k = 8t .. 8t + 7 of each group of its column, 16 bytes (8 in e4m3) of a row
// in global memory. They come straight into registers, right after the same
// groups of the stage before were used: a few rows stay in L1 and L2, and
// copying them through the ring cost one warp 730 cycles a stage, against the
// 390 of the copy bandwidth. Groups from `valid` on are left as they are.
template <bool kF16, bool kConst>
__device__ __forceinline__ void load_cols(const uint8_t* from, int valid, uint4& b0, uint4& b1) {
  const auto load = [](const uint8_t* p, uint4& b) {
    if constexpr (kF16) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      b.x = v.x;
      b.y = v.y;
    } else if constexpr (kConst) {
      b = __ldg(reinterpret_cast<const uint4*>(p));
    } else {  // written by this launch: not the read-only path
      b = *reinterpret_cast<const uint4*>(p);
    }
  };
  if (valid > 0) load(from, b0);
  if (valid > 1) load(from + (kF16 ? 32 : 64), b1);
}

// kG groups of 32 k of one 64-k step: 32 weight rows of this warp (two 16-row
// MMA tiles) times eight columns, kP parts per column value (b[group][part]);
// acc += scale * sum of every group.
// k order inside a group: thread t of a quad holds word t of each weight row
// (k = 8t .. 8t + 7) and the same eight values of its column; the two MMAs
// take code pairs (0, 1) and (2, 3), so both operands use one order.
// The scales of four rows and both groups come as one transposed ldmatrix
// whose addresses repeat two 16-byte runs.
template <int kP, bool kF16, int kG>
__device__ __forceinline__ void step_mma(uint32_t codes, uint32_t scales,
                                         const uint4 (&b)[2][kP], float (&acc)[2][4]) {
  uint32_t w[kG][4], sc[4];
#pragma unroll
  for (int g = 0; g < kG; ++g) ldmatrix_x4(codes + g * (kTileRows * 16), w[g]);
  ldmatrix_x4_trans(scales, sc);
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    uint4 v[kP];
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      v[p] = b[g][p];
      if constexpr (kF16)
        v[p] = make_uint4(e4m3_pair(b[g][p].x & 0xFFFFu), e4m3_pair(b[g][p].x >> 16),
                          e4m3_pair(b[g][p].y & 0xFFFFu), e4m3_pair(b[g][p].y >> 16));
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint32_t w0 = w[g][2 * mt], w1 = w[g][2 * mt + 1];
      float c[4];
      const uint32_t a0[4] = {code_pair<kF16>(w0, 0), code_pair<kF16>(w1, 0),
                              code_pair<kF16>(w0, 1), code_pair<kF16>(w1, 1)};
      const uint32_t a1[4] = {code_pair<kF16>(w0, 2), code_pair<kF16>(w1, 2),
                              code_pair<kF16>(w0, 3), code_pair<kF16>(w1, 3)};
      mma16816<kF16, true>(c, a0, v[kP - 1].x, v[kP - 1].y);
      mma16816<kF16, false>(c, a1, v[kP - 1].z, v[kP - 1].w);
#pragma unroll
      for (int p = kP - 2; p >= 0; --p) {  // smallest part first
        mma16816<kF16, false>(c, a0, v[p].x, v[p].y);
        mma16816<kF16, false>(c, a1, v[p].z, v[p].w);
      }
      const uint32_t pair = sc[2 * g + mt];
      const float s0 = __uint_as_float(pair << 16), s1 = __uint_as_float(pair & 0xFFFF0000u);
      acc[mt][0] = fmaf(s0, c[0], acc[mt][0]);
      acc[mt][1] = fmaf(s0, c[1], acc[mt][1]);
      acc[mt][2] = fmaf(s1, c[2], acc[mt][2]);
      acc[mt][3] = fmaf(s1, c[3], acc[mt][3]);
    }
  }
}

// One stage: its `valid` groups (1..4), then the columns of the next stage
// (`next_valid` groups at `next`, 0 for none) in the registers they leave.
template <bool kF16, bool kConst>
__device__ __forceinline__ void stage_mma(int valid, uint32_t codes, uint32_t scales,
                                          uint4 (&b)[4], const uint8_t* next, int next_valid,
                                          float (&acc)[2][4]) {
  const auto step = [&](uint32_t cs, uint32_t ss, int n, const uint4& b0, const uint4& b1) {
    const uint4 cols[2][1] = {{b0}, {b1}};
    if (n >= 2)
      step_mma<1, kF16, 2>(cs, ss, cols, acc);
    else if (n == 1)
      step_mma<1, kF16, 1>(cs, ss, cols, acc);
  };
  step(codes, scales, valid, b[0], b[1]);
  load_cols<kF16, kConst>(next, next_valid, b[0], b[1]);
  step(codes + kStepBytes, scales + kStepBytes, valid - 2, b[2], b[3]);
  load_cols<kF16, kConst>(next + (kF16 ? 64 : 128), next_valid - 2, b[2], b[3]);
}

// A stage with the kParts parts of every column value, part_bytes apart.
__device__ __forceinline__ void stage_mma_parts(int valid, uint32_t codes, uint32_t scales,
                                                const uint8_t* from, long long part_bytes,
                                                float (&acc)[2][4]) {
#pragma unroll 1
  for (int g0 = 0; g0 < valid; g0 += 2) {  // (the intermediate size is a multiple of 64)
    uint4 b[2][kParts];
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int p = 0; p < kParts; ++p)
        b[g][p] = *reinterpret_cast<const uint4*>(from + (g0 + g) * 64 + p * part_bytes);
    step_mma<kParts, false, 2>(codes, scales, b, acc);
    codes += kStepBytes;
    scales += kStepBytes;
  }
}

// ---------------------------------------------------------------- waits ---

__device__ __forceinline__ bool few_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         int* status, int where, long long timeout) {
  if (mbar_try_wait_sleep(bar, parity, 1000000)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait_sleep(bar, parity, 1000000)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > timeout) {
      *abort_flag = 1;
      atomicCAS(status, 0, 0x1000 | where);
      return false;
    }
  }
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
// sum over the warpgroups of four adjacent values
__device__ __forceinline__ float4 group_sum(const float* from, int stride) {
  const auto at = [&](int g) { return *reinterpret_cast<const float4*>(from + g * stride); };
  return add4(add4(at(0), at(1)), add4(at(2), at(3)));
}

__device__ __forceinline__ void epilogue_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kEpilogueThreads) : "memory");
}

// Arrive at a global counter after everything the epilogue warps wrote, and
// (returned to all of them) whether this was arrival number `last`.
__device__ __forceinline__ bool epilogue_arrive(int* counter, int last, int* flag, int etid) {
  epilogue_sync();
  if (etid == 0) {
    __threadfence();
    *flag = atomicAdd(counter, 1) == last;
    __threadfence();
  }
  epilogue_sync();
  return *flag != 0;
}

__device__ __forceinline__ void slot_next(int& slot, uint32_t& phase, int step, int slots) {
  slot += step;
  if (slot >= slots) {
    slot -= slots;
    phase ^= 1u;
  }
}

// The stages of one product, cut into equal runs: CTA b of `grid` owns
// [begin(b), begin(b + 1)), `base` stages each and one more for the first
// `extra` CTAs (the host keeps the total below 2^30).
struct Split {
  int stages;  // of one item
  int grid, base, extra;
  __device__ __forceinline__ Split(int items, int item_stages, int ctas) {
    const int total = items * item_stages;
    stages = item_stages;
    grid = min(ctas, total);
    base = total / grid;
    extra = total - base * grid;
  }
  __device__ __forceinline__ int begin(int b) const { return b * base + min(b, extra); }
  // the CTA that owns stage `at`
  __device__ __forceinline__ int owner(int at) const {
    const int longer = extra * (base + 1);
    return at < longer ? at / (base + 1) : extra + (at - longer) / base;
  }
};

}  // namespace

template <bool kFp8>
__global__ void __launch_bounds__(kFewThreads, 1) w4a16_moe_few_kernel(const FewParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const FewArgs& a = p.a;
  const FewSmem& sm = p.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows_cap = max_rows(a.tokens, a.topk);

  const uint32_t bar_w = smem_u32(smem), bar_e = bar_w + 8 * kMaxSlots;  // slots full, slots free
  const uint32_t bar_sf = bar_w + 16 * kMaxSlots, bar_se = bar_sf + 16;  // sums full, free
  const uint32_t bar_act = bar_se + 16;                                  // activation complete
  int* scalars = reinterpret_cast<int*>(smem + 16 * kMaxSlots + 48);
  volatile int* abort_flag = scalars;
  int* last_arrival = scalars + 1;
  int* num_chunks_p = scalars + 2;
  int* warp_sums = scalars + 4;  // [16]
  float* sums = reinterpret_cast<float*>(smem + sm.sums);
  int* s_ids = reinterpret_cast<int*>(smem + sm.ids);
  float* s_weights = reinterpret_cast<float*>(smem + sm.weights);
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem + sm.mask);
  int* s_base = reinterpret_cast<int*>(smem + sm.base);
  int* row_token = reinterpret_cast<int*>(smem + sm.row_token);
  float* row_weight = reinterpret_cast<float*>(smem + sm.row_weight);
  uint32_t* chunks = reinterpret_cast<uint32_t*>(smem + sm.chunks);
  float* s_xscales = reinterpret_cast<float*>(smem + sm.x_scales);
  const uint32_t ring = smem_u32(smem + sm.ring);

  int* status = reinterpret_cast<int*>(a.workspace);
  FewCounters* counters = reinterpret_cast<FewCounters*>(a.workspace + kStatusBytes);
  float* shares = reinterpret_cast<float*>(a.workspace + kStatusBytes + kCounterBytes);
  const size_t share = share_floats(a.tokens);
  uint16_t* act = reinterpret_cast<uint16_t*>(shares + 2 * kMaxCtas * share);

  // ---- setup: barriers, routing, the rows of every expert ----
  if (warp == kFewThreads / 32 - 1) {
    if (lane < sm.slots) {
      mbar_init(bar_w + 8 * lane, 1);
      mbar_init(bar_e + 8 * lane, 4);
    }
    if (lane < 2) {
      mbar_init(bar_sf + 8 * lane, kComputeWarps);
      mbar_init(bar_se + 8 * lane, kEpilogueWarps);
    }
    if (lane == 0) {
      mbar_init(bar_act, 1);
      *abort_flag = 0;
    }
    fence_mbar_init();
  }
  for (int e = tid; e < a.num_experts; e += kFewThreads) s_mask[e] = 0u;
  if (a.logits != nullptr) {
    for (int t = warp; t < a.tokens; t += kFewThreads / 32) {
      if (a.num_global <= 512)
        route_token<16>(a.logits, a.bf16_logits, t, a.num_global, a.topk, a.renormalize,
                        a.expert_offset, a.num_experts, s_ids, s_weights);
      else
        route_token<32>(a.logits, a.bf16_logits, t, a.num_global, a.topk, a.renormalize,
                        a.expert_offset, a.num_experts, s_ids, s_weights);
    }
  } else {
    for (int i = tid; i < rows_cap; i += kFewThreads) {
      s_ids[i] = a.topk_ids[i];
      s_weights[i] = a.topk_weights[i];
    }
  }
  if constexpr (kFp8) {
    const int n = a.tokens * ((a.hidden + kStageK - 1) / kStageK);
    for (int i = tid; i < n; i += kFewThreads) s_xscales[i] = a.x_scales[i];
  }
  __syncthreads();
  if (a.logits != nullptr && blockIdx.x == 0)
    for (int i = tid; i < rows_cap; i += kFewThreads) {
      a.topk_ids[i] = s_ids[i];
      a.topk_weights[i] = s_weights[i];
    }
  // bit t of an expert's mask: token t goes there
  for (int i = tid; i < rows_cap; i += kFewThreads) {
    const int e = s_ids[i];
    if (e >= 0 && e < a.num_experts) atomicOr(s_mask + e, 1u << (i / a.topk));
  }
  __syncthreads();
  // running sums over the experts of (rows, passes of up to eight rows):
  // thread i of the first 512 holds experts 2i and 2i + 1
  const auto rows_and_passes = [](uint32_t mask) {
    const uint32_t n = __popc(mask);
    return n | (n + kRowsPerPass - 1) / kRowsPerPass << 16;
  };
  uint32_t mine[2] = {0u, 0u}, own[2] = {0u, 0u}, incl = 0u;
  if (warp < kComputeWarps) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mine[i] = 2 * tid + i < a.num_experts ? s_mask[2 * tid + i] : 0u;
      own[i] = rows_and_passes(mine[i]);
    }
    incl = own[0] + own[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sums[warp] = static_cast<int>(incl);
  }
  __syncthreads();
  if (warp < kComputeWarps) {
    const uint32_t v = lane < kComputeWarps ? static_cast<uint32_t>(warp_sums[lane]) : 0u;
    const uint32_t all = __reduce_add_sync(0xffffffffu, v);
    uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0u) + incl - own[0] - own[1];
    if (tid == 0) *num_chunks_p = static_cast<int>(all >> 16);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 2 * tid + i, n = __popc(mine[i]);
      if (n > 0) {
        const int row = static_cast<int>(before & 0xFFFFu);
        int c = static_cast<int>(before >> 16);
        s_base[e] = row;
        // expert | rows - 1 << 10 | first row << 16
        for (int r = 0; r < n; r += kRowsPerPass)
          chunks[c++] = static_cast<uint32_t>(e) |
                        static_cast<uint32_t>(min(kRowsPerPass, n - r) - 1) << 10 |
                        static_cast<uint32_t>(row + r) << 16;
      }
      before += own[i];
    }
  }
  __syncthreads();
  // every pick finds its row: the expert's first row + the tokens before it;
  // the weight of an expert that a token names twice is the sum (both picks
  // write the same)
  for (int i = tid; i < rows_cap; i += kFewThreads) {
    const int e = s_ids[i];
    if (e < 0 || e >= a.num_experts) continue;
    const int tok = i / a.topk;
    const int row = s_base[e] + __popc(s_mask[e] & ((1u << tok) - 1u));
    float w = 0.f;
    for (int k = 0; k < a.topk; ++k)
      if (s_ids[tok * a.topk + k] == e) w += s_weights[tok * a.topk + k];
    row_token[row] = tok;
    row_weight[row] = w;
  }
  __syncthreads();

  const int num_chunks = *num_chunks_p;
  if (num_chunks == 0) {  // no row for this GPU's experts
    if (!a.accumulate)
      for (long long i = static_cast<long long>(blockIdx.x) * kFewThreads + tid;
           i < static_cast<long long>(a.tokens) * a.hidden;
           i += static_cast<long long>(gridDim.x) * kFewThreads)
        a.out[i] = 0.f;
    return;
  }
  // gate_up items: expert (pass) by expert, tile by tile; down items: tile by
  // tile, expert by expert
  const int steps0 = (a.hidden + kKStep - 1) / kKStep, steps1 = (a.inter + kKStep - 1) / kKStep;
  const int groups0 = a.hidden / kGroup, groups1 = a.inter / kGroup;
  const int tiles0 = a.inter / 64, tiles1 = (a.hidden + kTileRows - 1) / kTileRows;
  const Split gu(num_chunks * tiles0, (steps0 + 1) / 2, gridDim.x);
  const Split dn(num_chunks * tiles1, (steps1 + 1) / 2, gridDim.x);
  const int cta = blockIdx.x;
  const int gu_begin = cta < gu.grid ? gu.begin(cta) : 0, gu_end = cta < gu.grid ? gu.begin(cta + 1) : 0;
  const int dn_begin = cta < dn.grid ? dn.begin(cta) : 0, dn_end = cta < dn.grid ? dn.begin(cta + 1) : 0;
  const int gu_count = gu_end - gu_begin;

  if (warp >= kWarpWeights0 && warp < kWarpEpilogue0) {
    // ---- weight copies (one thread of each warp) ----
    if (lane == 0) {
      const uint64_t policy = policy_evict_first();
      const int first = warp - kWarpWeights0;
      int slot = first;
      uint32_t phase = 0;
      int next = first;  // stage of this CTA, over both products
      bool ok = true;
#pragma unroll
      for (int ph = 0; ph < 2; ++ph) {
        const int begin = ph == 0 ? gu_begin : dn_begin - gu_count;
        const int end = ph == 0 ? gu_end : dn_end;
        if (!ok || begin + next >= end) continue;
        const int S = ph == 0 ? gu.stages : dn.stages;
        const int steps = ph == 0 ? steps0 : steps1;
        const int inner_n = ph == 0 ? tiles0 : num_chunks;
        const int q = (begin + next) / S;
        int s = begin + next - q * S, outer = q / inner_n, inner = q - outer * inner_n;
        const uint8_t* base = ph == 0 ? a.gate_up : a.down;
        const long long expert_bytes = ph == 0 ? a.gate_up_expert_bytes : a.down_expert_bytes;
        const uint8_t* src = nullptr;
        bool fresh = true;
        for (; begin + next < end; next += kWeightWarps) {
          if (fresh) {
            const int c = ph == 0 ? outer : inner, tile = ph == 0 ? inner : outer;
            src = base + (chunks[c] & 1023u) * expert_bytes +
                  static_cast<long long>(tile) * steps * kStepBytes;
            fresh = false;
          }
          if (!few_wait(bar_e + 8 * slot, phase ^ 1u, abort_flag, status, kWhereRing,
                        a.timeout_cycles)) {
            ok = false;
            break;
          }
          const uint32_t bytes = min(2, steps - 2 * s) * kStepBytes;
          mbar_arrive_expect_tx(bar_w + 8 * slot, bytes);
          bulk_g2s(ring + slot * kWStage, src + static_cast<long long>(s) * kWStage, bytes,
                   bar_w + 8 * slot, policy);
          slot_next(slot, phase, kWeightWarps, sm.slots);
          s += kWeightWarps;
          while (s >= S) {
            s -= S;
            fresh = true;
            if (++inner == inner_n) {
              inner = 0;
              ++outer;
            }
          }
        }
      }
      if (!ok)  // copies in flight land before the CTA ends
        for (int u = first; u < next; u += kWeightWarps) {
          if (u < next - sm.slots) continue;
          const long long t0 = clock64();
          while (!mbar_try_wait(bar_w + 8 * (u % sm.slots), (u / sm.slots) & 1) &&
                 clock64() - t0 < kFewDrainCycles) {
          }
        }
    }
  } else if (warp < kComputeWarps) {
    // ---- compute: warpgroup `grp` takes the stages u % 4 == grp ----
    // After a wait gave up every warp still walks its stages (on whatever the
    // ring holds), so that the epilogue warps and the other CTAs meet all the
    // arrivals they count on.
    const int grp = warp >> 2;
    const int m0 = (warp & 3) * 32;  // this warp's weight rows in a tile
    const int g = lane >> 2, t = lane & 3;
    int slot = grp;                  // slot and phase of this group's next stage
    uint32_t phase = 0;
    bool live = true;
    uint32_t uses0 = 0, uses1 = 0;   // of the two sum buffers
    const uint32_t codes_at = (m0 + lane) * 16;
    // lane = (matrix, row): matrix m gives rows 16 (m & 1) .. + 15 of group
    // m >> 1; its eight addresses alternate between rows + 0 and rows + 8
    const uint32_t scales_at = kStepQBytes + ((lane >> 4) & 1) * (kTileRows * 2) +
                               (m0 + ((lane >> 3) & 1) * 16 + (lane & 1) * 8) * 2;
    const auto wait_sums = [&](uint32_t bar, uint32_t uses) {
      if (live)
        live = __all_sync(0xffffffffu, few_wait(bar, (uses & 1) ^ 1, abort_flag, status,
                                                kWhereSums, a.timeout_cycles));
    };
    const auto wait_stage = [&]() {
      if (live)
        live = __all_sync(0xffffffffu, few_wait(bar_w + 8 * slot, phase, abort_flag, status,
                                                kWhereData, a.timeout_cycles));
      return ring + slot * kWStage;
    };
    const auto free_stage = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_e + 8 * slot);
      slot_next(slot, phase, kGroups, sm.slots);
    };

    if (gu_count > 0) {
      const int S = gu.stages;
      // this lane's column of item q: row g of the pass (columns past the rows
      // repeat row 0 and are not used), from k = 8t on
      const auto item_cols = [&](int q) {
        const uint32_t ch = chunks[q / tiles0];
        const int n = static_cast<int>((ch >> 10) & 7u) + 1;
        const int tok = row_token[static_cast<int>(ch >> 16) + (g < n ? g : 0)];
        return static_cast<const uint8_t*>(a.x) +
               static_cast<long long>(tok) * a.hidden * (kFp8 ? 1 : 2) + t * (kFp8 ? 8 : 16);
      };
      constexpr int kStageBytes = kStageK * (kFp8 ? 1 : 2);
      uint4 b[4] = {};
      int at = gu_begin + grp;
      int next_q = at / S, next_s = at - next_q * S;  // item and stage of `at`
      const uint8_t* cols = nullptr;
      if (at < gu_end) {
        cols = item_cols(next_q);
        const uint8_t* from = cols + next_s * kStageBytes;
        load_cols<kFp8, true>(from, groups0 - 4 * next_s, b[0], b[1]);
        load_cols<kFp8, true>(from + kStageBytes / 2, groups0 - 4 * next_s - 2, b[2], b[3]);
      }
      const int q_end = (gu_end - 1) / S;
      for (int q = gu_begin / S; q <= q_end; ++q) {
        // item q: this group's stages of it, then its sums to the epilogue
        const float* xs0 = s_xscales;
        const float* xs1 = s_xscales;
        if constexpr (kFp8) {
          const uint32_t ch = chunks[q / tiles0];
          const int n1 = static_cast<int>((ch >> 10) & 7u);
          const int row0 = static_cast<int>(ch >> 16);
          xs0 += row_token[row0 + min(2 * t, n1)] * S;
          xs1 += row_token[row0 + min(2 * t + 1, n1)] * S;
        }
        float acc[2][4] = {};
        while (next_q == q && at < gu_end) {
          const int st = next_s, valid = groups0 - 4 * st;
          at += kGroups;
          next_s += kGroups;
          while (next_s >= S) {
            next_s -= S;
            ++next_q;
          }
          int next_valid = 0;
          if (at < gu_end) {
            if (next_q != q) cols = item_cols(next_q);
            next_valid = groups0 - 4 * next_s;
          }
          const uint8_t* next = cols + next_s * kStageBytes;
          const uint32_t base = wait_stage();
          if constexpr (kFp8) {
            // the rows' scales cover exactly one stage
            const float x0 = xs0[st], x1 = xs1[st];
            float part[2][4] = {};
            stage_mma<true, true>(valid, base + codes_at, base + scales_at, b, next, next_valid,
                                  part);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              acc[mt][0] = fmaf(x0, part[mt][0], acc[mt][0]);
              acc[mt][1] = fmaf(x1, part[mt][1], acc[mt][1]);
              acc[mt][2] = fmaf(x0, part[mt][2], acc[mt][2]);
              acc[mt][3] = fmaf(x1, part[mt][3], acc[mt][3]);
            }
          } else {
            stage_mma<false, true>(valid, base + codes_at, base + scales_at, b, next, next_valid,
                                   acc);
          }
          free_stage();
        }
        // [row of the pass][128] of this warpgroup, in the buffers by turns
        const int buf = (uses0 + uses1) & 1;
        wait_sums(bar_se + 8 * buf, buf ? uses1 : uses0);
        float* my = sums + buf * kItemSums + grp * (kRowsPerPass * kSumPitch) + m0 + g;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            my[(2 * t + (i & 1)) * kSumPitch + mt * 16 + (i >> 1) * 8] = acc[mt][i];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_sf + 8 * buf);
        if (buf)
          ++uses1;
        else
          ++uses0;
      }
    }
    if (dn_end > dn_begin) {
      const int S = dn.stages;
      // both gate_up buffers are read: the tile's sums take their place
      wait_sums(bar_se, uses0);
      wait_sums(bar_se + 8, uses1);
      if (live)
        live = __all_sync(0xffffffffu, few_wait(bar_act, 0, abort_flag, status, kWhereAct,
                                                a.timeout_cycles));
      float* my = sums + grp * (a.tokens * kSumPitch) + m0;
      // this lane's column of a pass of one or two rows, whose parts fill one
      // MMA's columns (part p of row r is column 2p + r), or else its row
      const auto pass_cols = [&](int c) {
        const uint32_t ch = chunks[c];
        const int n = static_cast<int>((ch >> 10) & 7u) + 1;
        const int row = n <= 2 ? g & (n - 1) : (g < n ? g : 0);
        const int part = n <= 2 && g >> 1 < kParts ? g >> 1 : 0;
        return reinterpret_cast<const uint8_t*>(act) +
               ((static_cast<long long>(ch >> 16) + row) * kParts + part) * a.inter * 2 + t * 16;
      };
      constexpr int kStageBytes = 2 * kStageK;
      uint4 b[4] = {};
      int at = dn_begin + ((grp - gu_count) & 3);
      int next_c = at / S, next_s = at - next_c * S;  // pass and stage of `at`
      next_c %= num_chunks;
      const uint8_t* cols = nullptr;
      if (at < dn_end) {
        cols = pass_cols(next_c);
        const uint8_t* from = cols + next_s * kStageBytes;
        load_cols<false, false>(from, groups1 - 4 * next_s, b[0], b[1]);
        load_cols<false, false>(from + kStageBytes / 2, groups1 - 4 * next_s - 2, b[2], b[3]);
      }
      const int tile_stages = num_chunks * S;
      const int tile_end = (dn_end - 1) / tile_stages;
      for (int tile = dn_begin / tile_stages; tile <= tile_end; ++tile) {
        // this group's stages of the tile, expert by expert: the passes' rows
        // are added to their tokens
        wait_sums(bar_se, uses0);
        for (int tok = 0; tok < a.tokens; ++tok) my[tok * kSumPitch + lane] = 0.f;
        __syncwarp();
        const int stop = min(dn_end, (tile + 1) * tile_stages);
        while (at < stop) {
          const uint32_t ch = chunks[next_c];
          const int n = static_cast<int>((ch >> 10) & 7u) + 1;
          const int row0 = static_cast<int>(ch >> 16);
          const bool packed = n <= 2;
          float acc[2][4] = {};
          bool more = true;  // own stages left in this pass
#pragma unroll 1
          while (more) {
            const int st = next_s, valid = groups1 - 4 * st;
            const uint8_t* here = cols;
            at += kGroups;
            next_s += kGroups;
            more = next_s < S && at < stop;
            int next_valid = 0;
            if (at < dn_end) {
              if (next_s >= S) {
                do {
                  next_s -= S;
                  if (++next_c == num_chunks) next_c = 0;
                } while (next_s >= S);
                cols = pass_cols(next_c);
              }
              next_valid = groups1 - 4 * next_s;
            }
            const uint8_t* next = cols + next_s * kStageBytes;
            const uint32_t base = wait_stage();
            if (packed) {
              stage_mma<false, false>(valid, base + codes_at, base + scales_at, b, next,
                                      next_valid, acc);
            } else {
              stage_mma_parts(min(4, valid), base + codes_at, base + scales_at,
                              here + st * kStageBytes, static_cast<long long>(a.inter) * 2, acc);
              load_cols<false, false>(next, next_valid, b[0], b[1]);
              load_cols<false, false>(next + kStageBytes / 2, next_valid - 2, b[2], b[3]);
            }
            free_stage();
          }
          if (packed) {
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float v = t < kParts ? acc[mt][i] : 0.f;
                v += __shfl_xor_sync(0xffffffffu, v, 2);  // (first + third part), second
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                acc[mt][i] = v;
              }
          }
          const int last = packed ? (t == 0 ? n : 0) : n;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 2 * t + i;
            if (r < last) {
              const float w = row_weight[row0 + r];
              float* dst = my + row_token[row0 + r] * kSumPitch + g;
#pragma unroll
              for (int mt = 0; mt < 2; ++mt) {
                dst[mt * 16] = fmaf(w, acc[mt][i], dst[mt * 16]);
                dst[mt * 16 + 8] = fmaf(w, acc[mt][2 + i], dst[mt * 16 + 8]);
              }
            }
          }
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(bar_sf);
        ++uses0;
      }
    }
  } else {
    // ---- epilogue warps: the items' sums to the activation, the tiles' to
    // the output; shares of cut items through the workspace ----
    const int etid = tid - 32 * kWarpEpilogue0;
    bool live = true;
    uint32_t items = 0;  // sums taken, the two buffers by turns
    if (gu_count > 0) {
      const int S = gu.stages;
      int q = gu_begin / S, at = gu_begin;
      int s0 = gu_begin - q * S;
      while (at < gu_end) {
        const int len = min(S - s0, gu_end - at);
        const int outer = q / tiles0, inner = q - outer * tiles0;
        const uint32_t ch = chunks[outer];
        const int n = static_cast<int>((ch >> 10) & 7u) + 1, row0 = static_cast<int>(ch >> 16);
        const bool whole = len == S;
        const int cta0 = gu.owner(q * S), cta1 = gu.owner(q * S + S - 1);
        const int buf = items & 1;
        if (live)
          live = __all_sync(0xffffffffu, few_wait(bar_sf + 8 * buf, (items >> 1) & 1, abort_flag,
                                                  status, kWhereSums, a.timeout_cycles));
        constexpr int kStride = kRowsPerPass * kSumPitch;
        const float* from0 = sums + buf * kItemSums;
        // act = silu(gate) * up of column c, row r, as three BF16 parts
        const auto put_act = [&](int c, int r, float gate, float up) {
          const float v = gate / (1.f + expf(-gate)) * up;
          uint16_t* dst =
              act + static_cast<long long>(row0 + r) * kParts * a.inter + inner * 64 + c;
          const uint32_t bits = __float_as_uint(v);
          if ((bits & 0x7F800000u) == 0x7F800000u) {  // infinity or NaN: one part
            dst[0] = static_cast<uint16_t>(bits >> 16 | ((bits & 0xFFFFu) != 0 ? 0x40u : 0u));
            dst[a.inter] = 0;
            dst[2 * a.inter] = 0;
          } else {
            const float r1 = v - __uint_as_float(bits & 0xFFFF0000u);
            const uint32_t bits1 = __float_as_uint(r1);
            const float r2 = r1 - __uint_as_float(bits1 & 0xFFFF0000u);
            dst[0] = static_cast<uint16_t>(bits >> 16);
            dst[a.inter] = static_cast<uint16_t>(bits1 >> 16);
            dst[2 * a.inter] = static_cast<uint16_t>(__float_as_uint(r2) >> 16);
          }
        };
        // thread = activation column; its gate and up rows of the tile
        const int c = etid, at_g = (c >> 4) * 32 + (c & 15);
        bool finish = whole;
        if (whole) {
          for (int r = 0; r < n; ++r) {
            const float* f = from0 + r * kSumPitch + at_g;
            const float gate = (f[0] + f[kStride]) + (f[2 * kStride] + f[3 * kStride]);
            f += 16;
            put_act(c, r, gate, (f[0] + f[kStride]) + (f[2 * kStride] + f[3 * kStride]));
          }
        } else {
          float4* dst =
              reinterpret_cast<float4*>(shares + (2 * cta + (cta == cta0 ? 1 : 0)) * share);
#pragma unroll 2
          for (int i = etid; i < n * (kTileRows / 4); i += kEpilogueThreads)
            __stcg(dst + i, group_sum(from0 + (i >> 5) * kSumPitch + (i & 31) * 4, kStride));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_se + 8 * buf);
        ++items;
        if (!whole) {
          // the CTA that arrives last adds the shares, in the CTAs' order
          finish = epilogue_arrive(&counters->item[0][cta0], cta1 - cta0, last_arrival, etid);
          if (finish) {
            float gate[kRowsPerPass] = {}, up[kRowsPerPass] = {};
#pragma unroll 2
            for (int b = cta0; b <= cta1; ++b) {
              const float* f = shares + (2 * b + (b == cta0 ? 1 : 0)) * share + at_g;
#pragma unroll
              for (int r = 0; r < kRowsPerPass; ++r)
                if (r < n) {
                  gate[r] += __ldcg(f + r * kTileRows);
                  up[r] += __ldcg(f + r * kTileRows + 16);
                }
            }
#pragma unroll
            for (int r = 0; r < kRowsPerPass; ++r)
              if (r < n) put_act(c, r, gate[r], up[r]);
          }
        }
        if (finish) {
          epilogue_sync();
          if (etid == 0) {
            __threadfence();
            atomicAdd(&counters->act_done, 1);
          }
        }
        at += len;
        s0 = 0;
        ++q;
      }
    }
    if (dn_end > dn_begin && etid == 0) {
      // every gate_up item of every CTA is out: the activation is complete
      const long long t0 = clock64();
      const int want = num_chunks * tiles0;
      while (true) {
        int v;
        asm volatile("ld.acquire.gpu.global.b32 %0, [%1];"
                     : "=r"(v)
                     : "l"(&counters->act_done)
                     : "memory");
        if (v >= want) {
          mbar_arrive(bar_act);
          break;
        }
        if (*abort_flag) break;
        if (clock64() - t0 > a.timeout_cycles) {
          *abort_flag = 1;
          atomicCAS(status, 0, 0x1000 | kWhereAct);
          break;
        }
      }
    }
    __syncwarp();
    if (dn_end > dn_begin) {
      const int tile_stages = num_chunks * dn.stages;
      const int stride = a.tokens * kSumPitch;
      uint32_t taken = (items + 1) >> 1;  // uses of the first buffer so far
      for (int at = dn_begin; at < dn_end; ++taken) {
        const int tile = at / tile_stages, tile0 = tile * tile_stages;
        const int cta0 = dn.owner(tile0), cta1 = dn.owner(tile0 + tile_stages - 1);
        const int h0 = tile * kTileRows;
        if (live)
          live = __all_sync(0xffffffffu, few_wait(bar_sf, taken & 1, abort_flag, status,
                                                  kWhereSums, a.timeout_cycles));
        float4* dst = reinterpret_cast<float4*>(shares + (2 * cta + (cta == cta0 ? 1 : 0)) * share);
        // four columns of a token (hidden is a multiple of 32)
        const auto put_out = [&](int i, float4 v) {
          const int h = h0 + (i & 31) * 4;
          if (h >= a.hidden) return;
          float4* o = reinterpret_cast<float4*>(
              a.out + static_cast<long long>(i >> 5) * a.hidden + h);
          *o = a.accumulate ? add4(*o, v) : v;
        };
        const int quads = a.tokens * (kTileRows / 4);
#pragma unroll 2
        for (int i = etid; i < quads; i += kEpilogueThreads) {
          const float4 v = group_sum(sums + (i >> 5) * kSumPitch + (i & 31) * 4, stride);
          if (cta0 != cta1)
            __stcg(dst + i, v);
          else
            put_out(i, v);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_se);
        if (cta0 != cta1 &&
            epilogue_arrive(&counters->item[1][cta0], cta1 - cta0, last_arrival, etid)) {
          // the shares in the CTAs' order, eight quads of a thread at a time
          for (int i0 = etid; i0 < quads; i0 += 8 * kEpilogueThreads) {
            float4 v[8] = {};
            for (int b = cta0; b <= cta1; ++b) {
              const float4* f = reinterpret_cast<const float4*>(
                  shares + (2 * b + (b == cta0 ? 1 : 0)) * share);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (i0 + j * kEpilogueThreads < quads)
                  v[j] = add4(v[j], __ldcg(f + i0 + j * kEpilogueThreads));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (i0 + j * kEpilogueThreads < quads) put_out(i0 + j * kEpilogueThreads, v[j]);
          }
        }
        at = min(dn_end, tile0 + tile_stages);
      }
    }
    // the last CTA out leaves the counters zero for the next call
    if (epilogue_arrive(&counters->exits, static_cast<int>(gridDim.x) - 1, last_arrival, etid)) {
      for (int i = etid; i < 2 * kMaxCtas; i += kEpilogueThreads) counters->item[0][i] = 0;
      if (etid == 0) {
        counters->act_done = 0;
        counters->exits = 0;
      }
    }
  }
}

size_t few_workspace_bytes(int tokens, int topk, int hidden, int inter) {
  (void)hidden;
  const int t = std::max(1, tokens);
  return kStatusBytes + kCounterBytes + 2 * kMaxCtas * share_floats(t) * sizeof(float) +
         static_cast<size_t>(max_rows(t, topk)) * kParts * inter * 2;
}

bool few_supported(int tokens, int topk, int num_experts, int hidden, int inter, bool fp8) {
  if (tokens == 0) return true;
  const long long rows = max_rows(tokens, topk);
  // the stage counts and the tile and column indexes stay inside 32 bits
  if (static_cast<long long>(hidden) > (1 << 20) || static_cast<long long>(inter) > (1 << 20))
    return false;
  if (fp8 && hidden > 16384) return false;  // the rows' scales stay in shared memory
  // passes (at most one a row) x tiles x stages of either product
  const long long stages = std::max<long long>(
      static_cast<long long>(inter / 64) * ((hidden + kStageK - 1) / kStageK),
      static_cast<long long>((hidden + kTileRows - 1) / kTileRows) *
          ((inter + kStageK - 1) / kStageK));
  if (rows * stages >= (1LL << 30)) return false;
  return rows <= 1024 && few_smem(tokens, topk, num_experts, hidden, fp8).slots >= kMinSlots;
}

cudaError_t launch_moe_few(const FewArgs& args, int sms, cudaStream_t stream) {
  FewParams p;
  p.a = args;
  p.s = few_smem(args.tokens, args.topk, args.num_experts, args.hidden, args.x_fp8 != 0);
  auto kernel = args.x_fp8 ? w4a16_moe_few_kernel<true> : w4a16_moe_few_kernel<false>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewMaxSmem);
  if (e != cudaSuccess) return e;
  kernel<<<std::min(sms, kMaxCtas), kFewThreads, p.s.total, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace w4a16
