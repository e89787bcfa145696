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
//     weight rows x 256 k (18432 packed bytes) and every CTA takes an equal,
//     contiguous run of them, first of gate_up, then of down, so that all SMs
//     read the same number of bytes whatever the number of experts;
//   * two threads copy the stages into a shared-memory ring (bulk copies);
//     they run through both products without waiting for the activation, so
//     the ring is full of down weights when the activation is complete;
//   * eight warps feed the codes to m16n8k16 MMAs of FP16 operands: a code in
//     bits 3 to 6 or 7 to 10 of a half word is the FP16 number q * 2^-21 or
//     q * 2^-17 (bits 0 to 9 of a subnormal and the lowest exponent bit above
//     them count on without a step), so a word of eight codes becomes four MMA
//     registers with two shifts and four ANDs. (In bits 0 to 7 one shift would
//     do, but the tensor core lines products up by their exponents, and a
//     subnormal's leading zeros are lost precision: 3.6e-6 of the output,
//     against 3e-7 with all codes in the highest bits, four shifts and 6 per
//     cent of the time.)
//     The 8 that every code is too large comes off as the number that a group's
//     sums start from, -8 times the columns, from two more MMAs a group.
//     Weights are the M side, the rows of an expert (at most four per pass over
//     its weights) the N side; the scale of a group of 32 is applied to the
//     group's FP32 sum, so no weight is rounded. The codes never leave
//     registers: through TMEM, as the tcgen05 kernel of the large batches needs
//     them, the same stream reaches 0.4 of the copy bandwidth, and as BF16
//     pairs q - 8 for BF16 MMAs 0.55. e4m3 MMAs, for which the code bytes would
//     do as they are, cost more: mma.sync converts their operands;
//   * the rows are put into FP16 first, times a power of two per block of 128
//     columns (a BF16 value fits exactly down to 2^-27 of its block's largest;
//     rows in e4m3 fit as they are); the FP32 activation goes into two FP16
//     parts per block of 64, 22 bits, each part a column of the MMA;
//   * two warps finish the items from shared memory while the others go on.
//
// An item (gate_up: one tile of one expert; down: one tile over all experts)
// may be cut between CTAs: each writes its FP32 share to the workspace and
// the CTA that arrives last adds the shares in order. Nothing is added with
// atomics, so the result depends only on the sizes, the routing and the number
// of CTAs.
//
// Measured, hidden 7168, top-8 of 384: 48 local experts of inter 2048, 32
// tokens: 134 us for 719 MB, 5.4 TB/s (0.79 of the copy rate); 384 experts of
// inter 256, 16 tokens: 81 us for 340 MB, 4.2 TB/s (0.62); 1 token 23.3 us, of
// which the 25 MB are 3.7. Inside the products the weights come at 6.2 TB/s
// (gate_up) and 5.3 (down, where the two columns of a row and the sums by token
// cost the compute warps more: tensor pipe 27 per cent of the whole call, ALU
// 40, issue slots 44); the rest is a chain of latencies: rows and routing 4.5
// us, lists 1.6, first copies 2.3, the activation's exchange 3 to 6.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "route_token.cuh"

namespace w4a16 {

namespace {

constexpr int kGroups = 4;                   // warpgroups; group g takes every fourth stage
constexpr int kGroupWarps = 2;               // of 64 weight rows each
constexpr int kComputeWarps = kGroupWarps * kGroups;
constexpr int kMt = 4;                       // 16-row MMA tiles of a warp
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
constexpr int kWStage = 4 * kStepBytes;      // packed bytes of a stage: four 64-k steps
constexpr int kStageK = 4 * kKStep;
constexpr int kHalfK = kStageK / 2;          // columns that a lane holds at a time
constexpr int kRowsPerPass = 4;              // rows of an expert per pass over its weights
constexpr int kActParts = 2;                 // FP16 parts of an activation value
constexpr float kPartScale = 2048.f;         // the second part is the rest times this
constexpr float kCodeScale = 2097152.f;      // a code is q * 2^-21
constexpr int kSumPitch = 132;               // FP32 sums [row][128 + 4]
constexpr int kMaxCtas = 192;
static_assert(kGroups % kWeightWarps == 0, "slots are shared out in turns");
constexpr int kMinSlots = kGroups;
constexpr int kMaxSlots = 8;  // 147 KB in flight (more measured slower)
constexpr int kFewMaxSmem = 232448;
constexpr long long kFewDrainCycles = 4000000000LL;

// waits that can give up (status word detail)
enum { kWhereRing = 0x21, kWhereData = 0x22, kWhereAct = 0x23, kWhereSums = 0x24,
       kWhereRows = 0x25 };

// Workspace: status words, counters, the CTAs' shares, the operands (Operand).
struct FewCounters {
  int act_done;               // finished gate_up items
  int exits;                  // CTAs that are through
  int rows_done;              // CTAs whose share of the rows is in FP16
  int pad;
  int item[2][kMaxCtas];      // arrivals at the item that a CTA begins and does not finish
};
constexpr size_t kCounterBytes = (sizeof(FewCounters) + 255) / 256 * 256;

__host__ __device__ inline int max_rows(int tokens, int topk) { return tokens * topk; }
__host__ __device__ inline size_t share_floats(int tokens) {
  return static_cast<size_t>(tokens > kRowsPerPass ? tokens : kRowsPerPass) * kTileRows;
}

// An MMA operand: `rows` rows of k FP16 values, and of every `block` columns
// the factor of the values (room for a row's factors in whole stages; those of
// blocks that the row does not have are never written, and not used).
struct Operand {
  size_t factors, bytes;  // byte offset, total
  int blocks;             // of a row
};
__host__ __device__ inline Operand operand(size_t rows, int k, int block) {
  Operand o;
  o.blocks = (k + kStageK - 1) / kStageK * (kStageK / block);
  o.factors = rows * k * 2;  // (k is a multiple of 32)
  o.bytes = (o.factors + rows * o.blocks * 4 + 15) / 16 * 16;
  return o;
}

// FP32 sums: two buffers of an item's sums by warpgroup (gate_up), or one of
// a tile's by warpgroup (down).
constexpr int kItemSums = kGroups * kRowsPerPass * kSumPitch;
inline int sum_floats(int tokens) { return std::max(2 * kItemSums, kGroups * tokens * kSumPitch); }

// Shared memory of a call, all offsets in bytes.
// Up to kLocalTokens tokens every CTA routes and converts all rows for itself,
// into shared memory; more are shared out, one exchange between the CTAs later.
constexpr int kLocalTokens = 2;
constexpr size_t kLocalBytes = 32 << 10;
inline bool few_local(int tokens, int hidden) {
  return tokens <= kLocalTokens && operand(tokens, hidden, kHalfK).bytes <= kLocalBytes;
}

struct FewSmem {
  int slots, ring;
  int local, rows;  // whether the rows lie here, and where
  int sums, ids, weights, mask, base, row_token, row_weight, chunks, total;
};
FewSmem few_smem(int tokens, int topk, int num_experts, int hidden) {
  FewSmem s;
  s.local = few_local(tokens, hidden);
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
  s.rows = take(s.local ? operand(tokens, hidden, kHalfK).bytes : 0);
  s.ring = at;
  // a multiple of the warpgroups and of the copy warps, so that each slot
  // belongs to one of each: otherwise one of them could come to a slot two
  // phases ahead of it, which a wait on the phase's parity cannot tell from done
  s.slots = std::min(kMaxSlots, (kFewMaxSmem - at) / kWStage) / kGroups * kGroups;
  s.total = at + s.slots * kWStage;
  return s;
}

struct FewParams {
  FewArgs a;
  FewSmem s;
};

// ------------------------------------------------------------------ MMA ---

// d = a . b + c
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
        "f"(c3));
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

// The power of two that takes a block whose largest |value| has these bits to
// [2^14, 2^15), inside FP16 (at most 2^127, for blocks that are nearly zero).
__device__ __forceinline__ float block_factor(uint32_t max_bits) {
  const int e = static_cast<int>(max_bits >> 23);
  return __uint_as_float(static_cast<uint32_t>(min(254, 268 - e)) << 23);
}

// Value k of a row as the MMAs take it: of every four codes of a row the last
// two lie four bits higher in their half words, times 16.
__device__ __forceinline__ float column_value(int k, float y) { return k & 2 ? y * 0.0625f : y; }

// The columns of half a stage in a lane's registers: thread t of a quad holds
// k = 8t .. 8t + 7 of each of the four groups of its MMA column. They come
// straight from L1 or L2, right after the same groups of the half before were
// used (a few rows stay there; copying them through the ring cost one warp 730
// cycles per 128 columns, against the 390 of the copy bandwidth). They were
// written by this launch: no read-only loads.
struct Cols {
  uint4 b[4];
};
__device__ __forceinline__ uint4 load16(const void* from) {
  return *reinterpret_cast<const uint4*>(from);
}

// The two groups of 32 k of a 64-k step: 64 weight rows of this warp (four 16-row
// MMA tiles) times eight columns, of which a thread keeps the even one or
// both; acc += scale * sum of every group.
// k order inside a group: thread t of a quad holds word t of each weight row
// (k = 8t .. 8t + 7) and the same eight values of its column; the first MMA
// takes k = 8t .. 8t + 3, the second the rest, so both operands use one order.
// The scales of four rows and both groups come as one transposed ldmatrix
// whose addresses repeat two 16-byte runs.
template <int kCols>
__device__ __forceinline__ void step_mma(uint32_t codes, uint32_t scales, const uint4& b0,
                                         const uint4& b1, float (&acc)[kMt][2 * kCols]) {
  constexpr uint32_t kLow = 0x00780078u, kHigh = 0x07800780u;
  const uint32_t minus8[4] = {0x80408040u, 0x80408040u, 0x84008400u, 0x84008400u};
  uint32_t w[2][kMt / 2][4], sc[kMt / 2][4];
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int h = 0; h < kMt / 2; ++h)
      ldmatrix_x4(codes + g * (kTileRows * 16) + h * 512, w[g][h]);
#pragma unroll
  for (int h = 0; h < kMt / 2; ++h) ldmatrix_x4_trans(scales + h * 64, sc[h]);
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const uint4 b = g == 0 ? b0 : b1;
    float i[4];
    mma16816(i, minus8, b.x, b.y, 0.f, 0.f, 0.f, 0.f);
    mma16816(i, minus8, b.z, b.w, i[0], i[1], i[2], i[3]);
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt) {
      const uint32_t w0 = w[g][mt >> 1][2 * (mt & 1)], w1 = w[g][mt >> 1][2 * (mt & 1) + 1];
      const uint32_t u0 = w0 << 3, u1 = w1 << 3, v0 = w0 >> 5, v1 = w1 >> 5;
      const uint32_t a0[4] = {u0 & kLow, u1 & kLow, u0 & kHigh, u1 & kHigh};
      const uint32_t a1[4] = {v0 & kLow, v1 & kLow, v0 & kHigh, v1 & kHigh};
      float c[4];
      mma16816(c, a0, b.x, b.y, i[0], i[1], i[2], i[3]);
      mma16816(c, a1, b.z, b.w, c[0], c[1], c[2], c[3]);
      const uint32_t pair = sc[mt >> 1][2 * g + (mt & 1)];
      const float s0 = __uint_as_float(pair << 16), s1 = __uint_as_float(pair & 0xFFFF0000u);
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        acc[mt][j] = fmaf(s0, c[j], acc[mt][j]);
        acc[mt][kCols + j] = fmaf(s1, c[2 + j], acc[mt][kCols + j]);
      }
    }
  }
}

// Half a stage: its `valid` groups (1..4, none for 0 or less), scaled by the
// factors of its two 64-k steps, then, into the registers they leave, the
// columns of the next half (`next_valid` groups at `next`).
// kCols: accumulated columns of a thread.
template <int kCols>
__device__ __forceinline__ void half_mma(int valid, uint32_t codes, uint32_t scales, Cols& x,
                                         float2 factor, const uint8_t* next, int next_valid,
                                         float (&acc)[kMt][2 * kCols]) {
  const auto step = [&](auto st, int n, int next_n) {
    constexpr int kS = decltype(st)::value;
    if (n > 0) {  // (a second group that the row does not have has scale 0)
      float part[kMt][2 * kCols] = {};
      step_mma<kCols>(codes + kS * kStepBytes, scales + kS * kStepBytes, x.b[2 * kS],
                         x.b[2 * kS + 1], part);
      // (a step that the row does not have has no factor either: what was read
      // for it is whatever the memory held, and 0 times that may be NaN)
      const float f = kS == 0 ? factor.x : factor.y;
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int i = 0; i < 2 * kCols; ++i) acc[mt][i] = fmaf(f, part[mt][i], acc[mt][i]);
    }
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    x.b[2 * kS] = next_n > 0 ? load16(next + kS * 128) : zero;
    x.b[2 * kS + 1] = next_n > 1 ? load16(next + kS * 128 + 64) : zero;
  };
  if (valid >= 4 && next_valid >= 4) {  // nearly always: no branch inside
    step(std::integral_constant<int, 0>(), 2, 2);
    step(std::integral_constant<int, 1>(), 2, 2);
  } else {
    step(std::integral_constant<int, 0>(), valid, next_valid);
    step(std::integral_constant<int, 1>(), valid - 2, next_valid - 2);
  }
}

// A stage in two halves; factor[h]: of the steps of half h.
template <int kCols>
__device__ __forceinline__ void stage_mma(int valid, uint32_t codes, uint32_t scales, Cols& x,
                                          float4 factor, const uint8_t* here, const uint8_t* next,
                                          int next_valid, float (&acc)[kMt][2 * kCols]) {
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    half_mma<kCols>(valid, codes, scales, x, make_float2(factor.x, factor.y),
                    h == 0 ? here + 2 * kHalfK : next, h == 0 ? valid - 4 : next_valid, acc);
    valid -= 4;
    codes += 2 * kStepBytes;
    scales += 2 * kStepBytes;
    factor.x = factor.z;
    factor.y = factor.w;
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

// Orders this thread's (and, behind a barrier, its CTA's) accesses before and
// after it for the whole GPU.
__device__ __forceinline__ void gpu_fence() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }

// Until the counter that other CTAs raise has reached `want`; false if the
// wait gave up.
__device__ __forceinline__ bool wait_count(const int* counter, int want, volatile int* abort_flag,
                                           int* status, int where, long long timeout) {
  const long long t0 = clock64();
  while (true) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
    if (v >= want) return true;
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
    gpu_fence();
    *flag = atomicAdd(counter, 1) == last;
    gpu_fence();
  }
  epilogue_sync();
  return *flag != 0;
}

// One warp of a CTA that has used the counters for the last time. The last CTA
// to say so leaves all of them zero for the next call, whatever it did itself:
// after a wait that gave up the CTAs may have read different routings.
__device__ __forceinline__ void leave_counters(FewCounters* counters, int lane) {
  int last = 0;
  if (lane == 0) last = atomicAdd(&counters->exits, 1) == static_cast<int>(gridDim.x) - 1;
  if (!__shfl_sync(0xffffffffu, last, 0)) return;
  for (int i = lane; i < 2 * kMaxCtas; i += 32) counters->item[0][i] = 0;
  if (lane == 0) {
    counters->act_done = 0;
    counters->rows_done = 0;
    counters->exits = 0;
  }
}

__device__ __forceinline__ void slot_next(int& slot, uint32_t& phase, int step, int slots) {
  slot += step;
  if (slot >= slots) {
    slot -= slots;
    phase ^= 1u;
  }
}

// The stages of one product, cut into equal runs: CTA b of `grid` owns
// [begin(b), begin(b + 1)), `base` units each and one more for the first
// `extra` CTAs (the host keeps the total below 2^30). A unit is a stage, or a
// whole item where items are so short (two stages for each warpgroup) that the
// exchange of shares, some 2.5 us, takes longer than they do.
constexpr int kWholeItem = 2 * kGroups;
struct Split {
  int stages;  // of one pass over an expert's tile
  int unit, grid, base, extra;
  // `items` items of item_stages stages
  __device__ __forceinline__ Split(int items, int item_stages, int pass_stages, int ctas) {
    stages = pass_stages;
    unit = item_stages <= kWholeItem ? item_stages : 1;
    const int total = items * (item_stages / unit);
    grid = min(ctas, total);
    base = total / grid;
    extra = total - base * grid;
  }
  __device__ __forceinline__ int begin(int b) const { return (b * base + min(b, extra)) * unit; }
  // the CTA that owns stage `at`
  __device__ __forceinline__ int owner(int at) const {
    const int u = at / unit, longer = extra * (base + 1);
    return u < longer ? u / (base + 1) : extra + (u - longer) / base;
  }
};

}  // namespace

__global__ void __launch_bounds__(kFewThreads, 1) w4a16_moe_few_kernel(const FewParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const FewArgs& a = p.a;
  const FewSmem& sm = p.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows_cap = max_rows(a.tokens, a.topk);

  const uint32_t bar_w = smem_u32(smem), bar_e = bar_w + 8 * kMaxSlots;  // slots full, slots free
  const uint32_t bar_sf = bar_w + 16 * kMaxSlots, bar_se = bar_sf + 16;  // sums full, free
  const uint32_t bar_act = bar_se + 16;  // activation complete
  int* scalars = reinterpret_cast<int*>(smem + 16 * kMaxSlots + 64);
  volatile int* abort_flag = scalars;
  int* last_arrival = scalars + 1;
  int* num_chunks_p = scalars + 2;
  int* warp_sums = scalars + 4;  // [16]
  uint32_t* block_top = reinterpret_cast<uint32_t*>(scalars + 20);  // [2][kRowsPerPass]
  volatile int* act_ready = scalars + 3;
  float* sums = reinterpret_cast<float*>(smem + sm.sums);
  int* s_ids = reinterpret_cast<int*>(smem + sm.ids);
  float* s_weights = reinterpret_cast<float*>(smem + sm.weights);
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem + sm.mask);
  int* s_base = reinterpret_cast<int*>(smem + sm.base);
  int* row_token = reinterpret_cast<int*>(smem + sm.row_token);
  float* row_weight = reinterpret_cast<float*>(smem + sm.row_weight);
  uint32_t* chunks = reinterpret_cast<uint32_t*>(smem + sm.chunks);
  const uint32_t ring = smem_u32(smem + sm.ring);

  int* status = reinterpret_cast<int*>(a.workspace);
  FewCounters* counters = reinterpret_cast<FewCounters*>(a.workspace + kStatusBytes);
  float* shares = reinterpret_cast<float*>(a.workspace + kStatusBytes + kCounterBytes);
  const size_t share = share_floats(a.tokens);
  // the two operands: the rows, and the activation's parts (row r, part p: row 2r + p)
  const Operand xo = operand(a.tokens, a.hidden, kHalfK);
  uint8_t* act_op = reinterpret_cast<uint8_t*>(shares + 2 * kMaxCtas * share) + xo.bytes;
  uint8_t* x_op = sm.local ? smem + sm.rows : act_op - xo.bytes;
  const Operand ao = operand(static_cast<size_t>(rows_cap) * kActParts, a.inter, kKStep);

  // ---- setup: barriers, routing, the rows of every expert ----
  if (warp == kFewThreads / 32 - 1) {
    if (lane < sm.slots) {
      mbar_init(bar_w + 8 * lane, 1);
      mbar_init(bar_e + 8 * lane, kGroupWarps);
    }
    if (lane < 2) {
      mbar_init(bar_sf + 8 * lane, kComputeWarps);
      mbar_init(bar_se + 8 * lane, kEpilogueWarps);
    }
    if (lane == 0) {
      mbar_init(bar_act, 1);
      *abort_flag = 0;
      *act_ready = 0;
    }
    fence_mbar_init();
  }
  for (int e = tid; e < a.num_experts; e += kFewThreads) s_mask[e] = 0u;
  grid_dependency_wait();  // what follows reads what earlier launches wrote
  grid_dependents_go();
  if (a.logits != nullptr && (sm.local || static_cast<int>(blockIdx.x) < a.tokens)) {
    // the logits of the (first) token that this CTA routes, into L1 meanwhile
    const int bytes = a.num_global * (a.bf16_logits ? 2 : 4);
    const uint8_t* row = static_cast<const uint8_t*>(a.logits) +
                         (sm.local ? 0 : static_cast<long long>(blockIdx.x) * bytes);
    if (tid * 128 < bytes) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + tid * 128));
  }
  // the rows into FP16, all of them or this CTA's share: sixteen lanes a block
  // of 128
  {
    constexpr int kHalves = kFewThreads / 16;
    const int half = tid >> 4, l16 = lane & 15;
    const int row_blocks = (a.hidden + kHalfK - 1) / kHalfK;  // of the input's scales too
    const int blocks = a.tokens * row_blocks;
    for (int b0 = sm.local ? 0 : blockIdx.x * kHalves; b0 < blocks;
         b0 += sm.local ? kHalves : gridDim.x * kHalves) {
      const int blk = min(b0 + half, blocks - 1);  // (the last ones may repeat a block)
      const int tok = blk / row_blocks, kb = blk - tok * row_blocks, k0 = kb * kHalfK + l16 * 8;
      const long long at = static_cast<long long>(tok) * a.hidden + k0;
      const bool in = k0 < a.hidden;
      float y[8];
      float out_factor;
      if (a.x_fp8) {
        uint2 v = make_uint2(0u, 0u);
        if (in) v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) + at));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t two = (i < 2 ? v.x : v.y) >> (i & 1) * 16 & 0xFFFFu;
          const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two),
                                                           __NV_E4M3);
          const float2 f = __half22float2(__half2(h));
          y[2 * i] = f.x;
          y[2 * i + 1] = f.y;
        }
        out_factor = __ldg(a.x_scales + blk);
      } else {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (in) v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + at));
        const uint32_t word[4] = {v.x, v.y, v.z, v.w};
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          top = max(top, max((word[i] & 0x7FFFu) << 16, word[i] & 0x7FFF0000u));
          y[2 * i] = __uint_as_float(word[i] << 16);
          y[2 * i + 1] = __uint_as_float(word[i] & 0xFFFF0000u);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float factor = block_factor(top);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= factor;
        out_factor = 1.f / factor;
      }
      uint32_t packed[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(column_value(2 * i, y[2 * i]),
                                            column_value(2 * i + 1, y[2 * i + 1]));
        packed[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if (in)
        *reinterpret_cast<uint4*>(x_op + at * 2) =
            make_uint4(packed[0], packed[1], packed[2], packed[3]);
      if (l16 == 0)
        reinterpret_cast<float*>(x_op + xo.factors)[tok * xo.blocks + kb] = out_factor;
    }
  }
  // the routing: of all tokens, or one CTA a token, so that a call of many
  // waits for one only
  int32_t* ids = sm.local ? s_ids : a.topk_ids;
  float* weights = sm.local ? s_weights : a.topk_weights;
  if (a.logits != nullptr)
    for (int t = sm.local ? 0 : blockIdx.x; t < a.tokens; t += sm.local ? 1 : gridDim.x)
      route_token_cta<kFewThreads / 32>(a.logits, a.bf16_logits, t, a.num_global, a.topk,
                                        a.renormalize, a.expert_offset, a.num_experts, ids,
                                        weights, sums);
  __syncthreads();
  if (!sm.local) {
    if (tid == 0) {
      gpu_fence();
      atomicAdd(&counters->rows_done, 1);
      wait_count(&counters->rows_done, gridDim.x, abort_flag, status, kWhereRows,
                 a.timeout_cycles);
    }
    __syncthreads();
  }
  if (!sm.local || a.logits == nullptr) {
    for (int i = tid; i < rows_cap; i += kFewThreads) {
      s_ids[i] = __ldcg(a.topk_ids + i);
      s_weights[i] = __ldcg(a.topk_weights + i);
    }
    __syncthreads();
  } else if (blockIdx.x == 0) {
    for (int i = tid; i < rows_cap; i += kFewThreads) {
      a.topk_ids[i] = s_ids[i];
      a.topk_weights[i] = s_weights[i];
    }
  }
  if (a.tokens == 1) {
    // one token: every local pick is a row and a pass of its own, in slot order
    if (warp == 0) {
      const int e = lane < a.topk ? s_ids[lane] : -1;
      const bool local = e >= 0 && e < a.num_experts;
      const uint32_t all = __ballot_sync(0xffffffffu, local);
      const int row = __popc(all & ((1u << lane) - 1u));
      if (local) {
        row_token[row] = 0;
        row_weight[row] = s_weights[lane];
        chunks[row] = static_cast<uint32_t>(e) | static_cast<uint32_t>(row) << 16;
      }
      if (lane == 0) *num_chunks_p = __popc(all);
    }
    __syncthreads();
  } else {
  // bit t of an expert's mask: token t goes there
  for (int i = tid; i < rows_cap; i += kFewThreads) {
    const int e = s_ids[i];
    if (e >= 0 && e < a.num_experts) atomicOr(s_mask + e, 1u << (i / a.topk));
  }
  __syncthreads();
  // running sums over the experts of (rows, passes of up to four rows):
  // thread i of the compute warps holds kOwn experts from kOwn * i on
  const auto rows_and_passes = [](uint32_t mask) {
    const uint32_t n = __popc(mask);
    return n | (n + kRowsPerPass - 1) / kRowsPerPass << 16;
  };
  constexpr int kOwn = 1024 / kComputeThreads;
  uint32_t mine[kOwn] = {}, own = 0u, incl = 0u;
  if (warp < kComputeWarps) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      mine[i] = kOwn * tid + i < a.num_experts ? s_mask[kOwn * tid + i] : 0u;
      own += rows_and_passes(mine[i]);
    }
    incl = own;
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
    uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0u) + incl - own;
    if (tid == 0) *num_chunks_p = static_cast<int>(all >> 16);
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int e = kOwn * tid + i, n = __popc(mine[i]);
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
      before += rows_and_passes(mine[i]);
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
  }

  const int num_chunks = *num_chunks_p;
  if (num_chunks == 0) {  // no row for this GPU's experts
    if (!a.accumulate)
      for (long long i = static_cast<long long>(blockIdx.x) * kFewThreads + tid;
           i < static_cast<long long>(a.tokens) * a.hidden;
           i += static_cast<long long>(gridDim.x) * kFewThreads)
        a.out[i] = 0.f;
    if (warp == 0) {
      gpu_fence();
      leave_counters(counters, lane);
    }
    return;
  }
  // gate_up items: expert (pass) by expert, tile by tile; down items: tile by
  // tile, expert by expert
  const int steps0 = (a.hidden + kKStep - 1) / kKStep, steps1 = (a.inter + kKStep - 1) / kKStep;
  const int groups0 = a.hidden / kGroup, groups1 = a.inter / kGroup;
  const int tiles0 = a.inter / 64, tiles1 = (a.hidden + kTileRows - 1) / kTileRows;
  const Split gu(num_chunks * tiles0, (steps0 + 3) / 4, (steps0 + 3) / 4, gridDim.x);
  const Split dn(tiles1, num_chunks * ((steps1 + 3) / 4), (steps1 + 3) / 4, gridDim.x);
  const int cta = blockIdx.x;
  const int gu_begin = cta < gu.grid ? gu.begin(cta) : 0, gu_end = cta < gu.grid ? gu.begin(cta + 1) : 0;
  const int dn_begin = cta < dn.grid ? dn.begin(cta) : 0, dn_end = cta < dn.grid ? dn.begin(cta + 1) : 0;
  const int gu_count = gu_end - gu_begin;

  if (warp >= kWarpWeights0 && warp < kWarpEpilogue0) {
    // ---- weight copies, by lane 0; the lanes bring the lines that the stage
    // will meet into L1: four lines of four rows, or, once the activation is
    // complete, of four rows' two parts ----
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
      const uint8_t* line = nullptr;
      bool fresh = true;
      for (; begin + next < end; next += kWeightWarps) {
        if (fresh) {
          const uint32_t ch = chunks[ph == 0 ? outer : inner];
          const int tile = ph == 0 ? inner : outer;
          src = base + (ch & 1023u) * expert_bytes +
                static_cast<long long>(tile) * steps * kStepBytes;
          const int last = static_cast<int>(ch >> 10 & 7u), row0 = static_cast<int>(ch >> 16);
          line = ph == 0 ? x_op + static_cast<long long>(row_token[row0 + min(lane >> 2 & 3, last)]) *
                                      a.hidden * 2
                         : act_op + (static_cast<long long>(row0 + min(lane >> 3, last)) * kActParts +
                                     (lane >> 2 & 1)) *
                                        a.inter * 2;
          line += (lane & 3) * 128;
          fresh = false;
        }
        if (!__all_sync(0xffffffffu, few_wait(bar_e + 8 * slot, phase ^ 1u, abort_flag, status,
                                              kWhereRing, a.timeout_cycles))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const uint32_t bytes = min(4, steps - 4 * s) * kStepBytes;
          mbar_arrive_expect_tx(bar_w + 8 * slot, bytes);
          bulk_g2s(ring + slot * kWStage, src + static_cast<long long>(s) * kWStage, bytes,
                   bar_w + 8 * slot, policy);
        }
        if ((ph == 0 ? lane < 16 && !sm.local : *act_ready != 0) &&
            s * (2 * kStageK) + (lane & 3) * 128 < 2 * (ph == 0 ? a.hidden : a.inter))
          asm volatile("prefetch.global.L1 [%0];" ::"l"(line + s * (2 * kStageK)));
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
    if (!ok && lane == 0)  // copies in flight land before the CTA ends
      for (int u = first; u < next; u += kWeightWarps) {
        if (u < next - sm.slots) continue;
        const long long t0 = clock64();
        while (!mbar_try_wait(bar_w + 8 * (u % sm.slots), (u / sm.slots) & 1) &&
               clock64() - t0 < kFewDrainCycles) {
        }
      }
  } else if (warp < kComputeWarps) {
    // ---- compute: warpgroup `grp` takes the stages u % 4 == grp ----
    // After a wait gave up every warp still walks its stages (on whatever the
    // ring holds), so that the epilogue warps and the other CTAs meet all the
    // arrivals they count on.
    const int grp = warp / kGroupWarps;
    const int m0 = (warp % kGroupWarps) * 64;  // this warp's weight rows in a tile
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
      // thread t of a quad accumulates row t of the pass, as MMA column 2t
      // (column 2t + 1 is a copy; rows past the last repeat it)
      const auto token_of = [&](int q, int r) {
        const uint32_t ch = chunks[q / tiles0];
        return row_token[static_cast<int>(ch >> 16) + min(r, static_cast<int>(ch >> 10 & 7u))];
      };
      const uint8_t* cols = nullptr;   // from k = 8t on
      const float* factors = nullptr;
      const auto point = [&](int q) {
        cols = x_op + static_cast<long long>(token_of(q, g >> 1)) * a.hidden * 2 + t * 16;
        const int tok = token_of(q, t);
        factors = reinterpret_cast<const float*>(x_op + xo.factors) + tok * xo.blocks;
      };
      Cols x = {};
      float2 next_factor = make_float2(0.f, 0.f);  // of both halves
      int at = gu_begin + grp;
      int next_q = at / S, next_s = at - next_q * S;  // item and stage of `at`
      if (at < gu_end) {
        point(next_q);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < groups0 - 8 * next_s) x.b[i] = load16(cols + next_s * (2 * kStageK) + i * 64);
        next_factor = *reinterpret_cast<const float2*>(factors + 2 * next_s);
      }
      const int q_end = (gu_end - 1) / S;
      for (int q = gu_begin / S; q <= q_end; ++q) {
        // item q: this group's stages of it, then its sums to the epilogue
        float acc[kMt][2] = {};
#pragma unroll 1
        while (next_q == q && at < gu_end) {
          const int valid = groups0 - 8 * next_s;
          const uint8_t* here = cols + next_s * (2 * kStageK);
          at += kGroups;
          next_s += kGroups;
          while (next_s >= S) {
            next_s -= S;
            ++next_q;
          }
          // (behind the last stage the same columns come again, unused: a
          // branch of its own would be met with its instructions not there)
          int next_valid = valid;
          const uint8_t* next = here;
          const float2 factor = next_factor;
          if (at < gu_end) {
            if (next_q != q) point(next_q);
            next_valid = groups0 - 8 * next_s;
            next = cols + next_s * (2 * kStageK);
            next_factor = *reinterpret_cast<const float2*>(factors + 2 * next_s);
          }
          const uint32_t base = wait_stage();
          stage_mma<1>(valid, base + codes_at, base + scales_at, x,
                       make_float4(factor.x, factor.x, factor.y, factor.y), here, next,
                       next_valid, acc);
          free_stage();
        }
        // [row of the pass][128] of this warpgroup, in the buffers by turns
        const int buf = (uses0 + uses1) & 1;
        wait_sums(bar_se + 8 * buf, buf ? uses1 : uses0);
        float* my = sums + buf * kItemSums + grp * (kRowsPerPass * kSumPitch) + t * kSumPitch + m0 + g;
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) my[mt * 16 + h * 8] = acc[mt][h] * kCodeScale;
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
      // thread t of a quad accumulates row t of the pass, its two parts as MMA
      // columns 2t and 2t + 1 (rows past the last repeat it)
      const uint8_t* cols = nullptr;  // from k = 8t on
      const float* factors = nullptr;
      const auto point = [&](int c) {
        const uint32_t ch = chunks[c];
        const int last = static_cast<int>(ch >> 10 & 7u), row0 = static_cast<int>(ch >> 16);
        const long long part_row = (row0 + min(g >> 1, last)) * kActParts + (g & 1);
        cols = act_op + part_row * a.inter * 2 + t * 16;
        const long long first = (row0 + min(t, last)) * kActParts;
        factors = reinterpret_cast<const float*>(act_op + ao.factors) + first * ao.blocks;
      };
      Cols x = {};
      float4 next_factor = make_float4(0.f, 0.f, 0.f, 0.f);  // of the four 64-k steps
      int at = dn_begin + ((grp - gu_count) & 3);
      int next_c = at / S, next_s = at - next_c * S;  // pass and stage of `at`
      next_c %= num_chunks;
      if (at < dn_end) {
        point(next_c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < groups1 - 8 * next_s) x.b[i] = load16(cols + next_s * (2 * kStageK) + i * 64);
        next_factor = *reinterpret_cast<const float4*>(factors + 4 * next_s);
      }
      const int tile_stages = num_chunks * S;
      const int tile_end = (dn_end - 1) / tile_stages;
      for (int tile = dn_begin / tile_stages; tile <= tile_end; ++tile) {
        // this group's stages of the tile, expert by expert: the passes' rows
        // are added to their tokens
        wait_sums(bar_se, uses0);
        for (int tok = 0; tok < a.tokens; ++tok) my[tok * kSumPitch + lane] = my[tok * kSumPitch + 32 + lane] = 0.f;
        __syncwarp();
        const int stop = min(dn_end, (tile + 1) * tile_stages);
        while (at < stop) {
          const uint32_t ch = chunks[next_c];
          const int last = static_cast<int>(ch >> 10 & 7u), row = static_cast<int>(ch >> 16) + t;
          float acc[kMt][4] = {};
          bool more = true;  // own stages left in this pass
#pragma unroll 1
          while (more) {
            const int valid = groups1 - 8 * next_s;
            const uint8_t* here = cols + next_s * (2 * kStageK);
            at += kGroups;
            next_s += kGroups;
            more = next_s < S && at < stop;
            int next_valid = valid;
            const uint8_t* next = here;
            const float4 factor = next_factor;
            if (at < dn_end) {
              if (next_s >= S) {
                do {
                  next_s -= S;
                  if (++next_c == num_chunks) next_c = 0;
                } while (next_s >= S);
                point(next_c);
              }
              next_valid = groups1 - 8 * next_s;
              next = cols + next_s * (2 * kStageK);
              next_factor = *reinterpret_cast<const float4*>(factors + 4 * next_s);
            }
            const uint32_t base = wait_stage();
            stage_mma<2>(valid, base + codes_at, base + scales_at, x, factor, here, next,
                         next_valid, acc);
            free_stage();
          }
          if (t <= last) {
            const float w = row_weight[row] * kCodeScale;
            float* dst = my + row_token[row] * kSumPitch + g;
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float v = fmaf(acc[mt][2 * h + 1], 1.f / kPartScale, acc[mt][2 * h]);
                dst[mt * 16 + h * 8] = fmaf(w, v, dst[mt * 16 + h * 8]);
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
    const auto leave = [&]() {
      if (etid < 32) leave_counters(counters, etid);
    };
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
        // act = silu(gate) * up of column c and the pass's rows, as two FP16
        // parts, in the power of two of the block of 64 columns
        const auto put_act = [&](int c, const float (&gate)[kRowsPerPass],
                                 const float (&up)[kRowsPerPass]) {
          float v[kRowsPerPass];
#pragma unroll
          for (int r = 0; r < kRowsPerPass; ++r)
            if (r < n) {
              v[r] = gate[r] / (1.f + expf(-gate[r])) * up[r];
              const uint32_t top =
                  __reduce_max_sync(0xffffffffu, __float_as_uint(v[r]) & 0x7FFFFFFFu);
              if (lane == 0) block_top[(etid >> 5) * kRowsPerPass + r] = top;
            }
          epilogue_sync();
#pragma unroll
          for (int r = 0; r < kRowsPerPass; ++r)
            if (r < n) {
              const float factor = block_factor(max(block_top[r], block_top[kRowsPerPass + r]));
              const float y = v[r] * factor;
              const __half hi = __float2half_rn(y);
              // (0 beside an infinity or a NaN)
              float rest = (y - __half2float(hi)) * kPartScale;
              if (!(fabsf(y) < INFINITY)) rest = 0.f;
              const __half value[kActParts] = {hi, __float2half_rn(rest)};
              const long long row = static_cast<long long>(row0 + r) * kActParts;
#pragma unroll
              for (int p = 0; p < kActParts; ++p) {
                reinterpret_cast<__half*>(act_op)[(row + p) * a.inter + inner * 64 + c] =
                    __float2half_rn(column_value(c, __half2float(value[p])));
              }
              if (etid == 0)
                reinterpret_cast<float*>(act_op + ao.factors)[row * ao.blocks + inner] =
                    1.f / factor;
            }
        };
        // thread = activation column; its gate and up rows of the tile
        const int c = etid, at_g = (c >> 4) * 32 + (c & 15);
        bool finish = whole;
        float gate[kRowsPerPass] = {}, up[kRowsPerPass] = {};
        if (whole) {
#pragma unroll
          for (int r = 0; r < kRowsPerPass; ++r)
            if (r < n) {
              const float* f = from0 + r * kSumPitch + at_g;
              gate[r] = (f[0] + f[kStride]) + (f[2 * kStride] + f[3 * kStride]);
              f += 16;
              up[r] = (f[0] + f[kStride]) + (f[2 * kStride] + f[3 * kStride]);
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
            // (four at a time, so that a trip to L2 brings four)
            for (int b0 = cta0; b0 <= cta1; b0 += 4) {
              float part[4][kRowsPerPass][2];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int b = b0 + j;
                const float* f = shares + (2 * b + (b == cta0 ? 1 : 0)) * share + at_g;
#pragma unroll
                for (int r = 0; r < kRowsPerPass; ++r) {
                  const bool in = b <= cta1 && r < n;
                  part[j][r][0] = in ? __ldcg(f + r * kTileRows) : 0.f;
                  part[j][r][1] = in ? __ldcg(f + r * kTileRows + 16) : 0.f;
                }
              }
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < kRowsPerPass; ++r) {
                  gate[r] += part[j][r][0];
                  up[r] += part[j][r][1];
                }
            }
          }
        }
        if (finish) {
          put_act(c, gate, up);
          epilogue_sync();
          if (etid == 0) {
            gpu_fence();
            atomicAdd(&counters->act_done, 1);
          }
        }
        at += len;
        s0 = 0;
        ++q;
      }
    }
    // every gate_up item of every CTA is out: the activation is complete
    if (dn_end > dn_begin && etid == 0 &&
        wait_count(&counters->act_done, num_chunks * tiles0, abort_flag, status, kWhereAct,
                   a.timeout_cycles)) {
      *act_ready = 1;
      mbar_arrive(bar_act);
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
        const int next_at = min(dn_end, tile0 + tile_stages);
        const bool join = cta0 != cta1 && epilogue_arrive(&counters->item[1][cta0], cta1 - cta0,
                                                          last_arrival, etid);
        if (next_at == dn_end) leave();
        if (join) {
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
        at = next_at;
      }
    }
    if (dn_end == dn_begin) leave();
  }
}

size_t few_workspace_bytes(int tokens, int topk, int hidden, int inter) {
  const int t = std::max(1, tokens);
  const size_t rows = max_rows(t, topk);
  return kStatusBytes + kCounterBytes + 2 * kMaxCtas * share_floats(t) * sizeof(float) +
         operand(t, hidden, kHalfK).bytes + operand(rows * kActParts, inter, kKStep).bytes;
}

bool few_supported(int tokens, int topk, int num_experts, int hidden, int inter) {
  if (tokens == 0) return true;
  const long long rows = max_rows(tokens, topk);
  // the stage counts and the tile and column indexes stay inside 32 bits
  if (static_cast<long long>(hidden) > (1 << 20) || static_cast<long long>(inter) > (1 << 20))
    return false;
  // passes (at most one a row) x tiles x stages of either product
  const long long stages = std::max<long long>(
      static_cast<long long>(inter / 64) * ((hidden + kStageK - 1) / kStageK),
      static_cast<long long>((hidden + kTileRows - 1) / kTileRows) *
          ((inter + kStageK - 1) / kStageK));
  if (rows * stages >= (1LL << 30)) return false;
  return rows <= 1024 && few_smem(tokens, topk, num_experts, hidden).slots >= kMinSlots;
}

cudaError_t launch_moe_few(const FewArgs& args, int sms, cudaStream_t stream) {
  FewParams p;
  p.a = args;
  p.s = few_smem(args.tokens, args.topk, args.num_experts, args.hidden);
  const cudaError_t e = cudaFuncSetAttribute(
      w4a16_moe_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewMaxSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(w4a16_moe_few_kernel, std::min(sms, kMaxCtas), kFewThreads,
                          static_cast<size_t>(p.s.total), 1, stream, p);
}

}  // namespace w4a16
