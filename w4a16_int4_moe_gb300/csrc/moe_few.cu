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
//   * one thread copies the stages into a shared-memory ring (bulk copies);
//     it runs through both products without waiting for the activation, so
//     the ring is full of down weights when the activation is complete;
//   * sixteen warps turn the codes into 16-bit integers in registers and feed
//     them to m16n8k16 MMAs: weights are the M side, the rows of an expert
//     (at most eight per pass over its weights) the N side. q - 8 is exact in
//     16 bits; the scale of a group of 32 is applied to the group's FP32 sum,
//     so no weight is rounded. The dequantised weights never leave registers:
//     through TMEM, as the tcgen05 kernel of the large batches needs them,
//     the same stream reaches 0.4 of the copy bandwidth;
//   * the activation is handed to the second product as three BF16 parts whose
//     sum is the FP32 value (each part cuts off 8 bits), three MMAs into one
//     accumulator.
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
constexpr int kFewThreads = kComputeThreads + 64;  // + the weight warp and the row warp
constexpr int kWStage = 2 * kStepBytes;      // packed bytes of a stage: two 64-k steps
constexpr int kStageK = 2 * kKStep;
constexpr int kRowsPerPass = 8;              // rows of an expert per pass over its weights (MMA N)
constexpr int kParts = 3;                    // BF16 parts of an activation value
// Row pitches in a ring slot. A quad reads 64 (e4m3: 32) adjacent bytes of a
// row; these pitches put the rows of one shared-memory wavefront on different
// banks.
constexpr int kRowPitch = 2 * kStageK + 64;
constexpr int kRowPitchFp8 = kStageK + 32;
constexpr int kSumPitch = 132;               // FP32 sums [row][128 + 4]
constexpr int kMaxCtas = 192;
constexpr int kMinSlots = 4;
constexpr int kMaxSlots = 24;
constexpr int kFewMaxSmem = 232448;
constexpr long long kFewDrainCycles = 4000000000LL;

// waits that can give up (status word detail)
enum { kWhereRing = 0x21, kWhereRows = 0x22, kWhereData = 0x23, kWhereAct = 0x24 };

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

// Shared memory of a call, all offsets in bytes.
struct FewSmem {
  int slots, slot_bytes, rows_at;
  int sums, ids, weights, mask, row_token, row_weight, chunks, x_scales, total;
};
FewSmem few_smem(int tokens, int topk, int num_experts, int hidden, bool fp8) {
  FewSmem s;
  const int rows = max_rows(tokens, topk);
  const int n8 = std::min(tokens, kRowsPerPass);
  int at = 1024;  // barriers and scalars
  auto take = [&at](size_t bytes) {
    const int here = at;
    at += static_cast<int>((bytes + 127) / 128 * 128);
    return here;
  };
  s.sums = take(sizeof(float) * kGroups * std::max(tokens, kRowsPerPass) * kSumPitch);
  s.ids = take(4 * static_cast<size_t>(rows));
  s.weights = take(4 * static_cast<size_t>(rows));
  s.mask = take(4 * static_cast<size_t>(num_experts));
  s.row_token = take(4 * static_cast<size_t>(rows));
  s.row_weight = take(4 * static_cast<size_t>(rows));
  s.chunks = take(4 * static_cast<size_t>(rows));
  s.x_scales = take(fp8 ? 4 * static_cast<size_t>(tokens) * ((hidden + 127) / 128) : 0);
  s.rows_at = at;
  s.slot_bytes = kWStage + kParts * n8 * kRowPitch;
  s.slots = std::min(kMaxSlots, (kFewMaxSmem - at) / s.slot_bytes);
  s.total = at + s.slots * s.slot_bytes;
  return s;
}

struct FewParams {
  FewArgs a;
  FewSmem s;
};

// ------------------------------------------------------------------ MMA ---

template <bool kF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kF16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
}

// Codes 2i and 2i + 1 of a packed word as the pair (q - 8, q - 8): the nibble
// becomes the low mantissa bits of 128 (BF16) or 1024 (FP16), the difference
// to 136 or 1032 is exact.
template <bool kF16>
__device__ __forceinline__ uint32_t code_pair(uint32_t word, int i) {
  constexpr uint32_t kBase = kF16 ? 0x64006400u : 0x43004300u;
  constexpr uint32_t kZero = kF16 ? 0x64086408u : 0x43084308u;
  uint32_t v = ((word >> (4 * i)) & 0x000F000Fu) | kBase;
  uint32_t r;
  if constexpr (kF16)
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(kZero));
  else
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(kZero));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float lds_bf16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(r)
      : "r"(two));
  return r;
}

// One group of 32 k: 32 weight rows of this warp (two 16-row MMA tiles) times
// up to eight rows; acc += scale * sum.
// k order inside the group: thread t of a quad holds word t of each weight
// row (k = 8t .. 8t + 7) and the same eight values of its row of x; the two
// MMAs take code pairs (0, 1) and (2, 3), so both operands use one order.
template <int kP, bool kF16>
__device__ __forceinline__ void group_mma(uint32_t codes, uint32_t scales, uint32_t row,
                                          uint32_t part_bytes, float (&acc)[2][4]) {
  uint32_t w[4];
  ldmatrix_x4(codes, w);
  uint4 b[kP];
#pragma unroll
  for (int p = 0; p < kP; ++p) {
    if constexpr (kF16) {
      const uint2 v = lds64(row);
      b[p] = make_uint4(e4m3_pair(v.x & 0xFFFFu), e4m3_pair(v.x >> 16), e4m3_pair(v.y & 0xFFFFu),
                        e4m3_pair(v.y >> 16));
    } else {
      b[p] = lds128(row + p * part_bytes);
    }
  }
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    float c[4] = {0.f, 0.f, 0.f, 0.f};
    const uint32_t a0[4] = {code_pair<kF16>(w[2 * mt], 0), code_pair<kF16>(w[2 * mt + 1], 0),
                            code_pair<kF16>(w[2 * mt], 1), code_pair<kF16>(w[2 * mt + 1], 1)};
    const uint32_t a1[4] = {code_pair<kF16>(w[2 * mt], 2), code_pair<kF16>(w[2 * mt + 1], 2),
                            code_pair<kF16>(w[2 * mt], 3), code_pair<kF16>(w[2 * mt + 1], 3)};
#pragma unroll
    for (int p = kP - 1; p >= 0; --p) {  // smallest part first
      mma16816<kF16>(c, a0, b[p].x, b[p].y);
      mma16816<kF16>(c, a1, b[p].z, b[p].w);
    }
    const float s0 = lds_bf16(scales + mt * 32), s1 = lds_bf16(scales + mt * 32 + 16);
    acc[mt][0] = fmaf(s0, c[0], acc[mt][0]);
    acc[mt][1] = fmaf(s0, c[1], acc[mt][1]);
    acc[mt][2] = fmaf(s1, c[2], acc[mt][2]);
    acc[mt][3] = fmaf(s1, c[3], acc[mt][3]);
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

__device__ __forceinline__ void compute_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kComputeThreads) : "memory");
}

__device__ __forceinline__ void slot_next(int& slot, uint32_t& phase, int step, int slots) {
  slot += step;
  if (slot >= slots) {
    slot -= slots;
    phase ^= 1u;
  }
}

// The stages of one product: `items` items of `stages` stages; CTA b of `grid`
// owns [begin(b), begin(b + 1)).
struct Split {
  int stages;
  long long total;
  int grid;
  __device__ __forceinline__ long long begin(int b) const {
    return b >= grid ? total : static_cast<long long>(b) * total / grid;
  }
  // the CTA that owns stage `at`: the last one that begins at or before it
  __device__ __forceinline__ int owner(long long at) const {
    return static_cast<int>(((at + 1) * grid - 1) / total);
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

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);  // weights full, rows full, empty
  const uint32_t bar_w = smem_u32(bars), bar_x = bar_w + 8 * kMaxSlots,
                 bar_e = bar_w + 16 * kMaxSlots;
  int* scalars = reinterpret_cast<int*>(smem + 24 * kMaxSlots);
  volatile int* abort_flag = scalars;
  int* last_arrival = scalars + 1;
  int* num_chunks_p = scalars + 2;
  int* warp_sums = scalars + 4;  // [16]
  float* sums = reinterpret_cast<float*>(smem + sm.sums);
  int* s_ids = reinterpret_cast<int*>(smem + sm.ids);
  float* s_weights = reinterpret_cast<float*>(smem + sm.weights);
  uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem + sm.mask);
  int* row_token = reinterpret_cast<int*>(smem + sm.row_token);
  float* row_weight = reinterpret_cast<float*>(smem + sm.row_weight);
  uint32_t* chunks = reinterpret_cast<uint32_t*>(smem + sm.chunks);
  float* s_xscales = reinterpret_cast<float*>(smem + sm.x_scales);
  const uint32_t ring = smem_u32(smem + sm.rows_at);

  int* status = reinterpret_cast<int*>(a.workspace);
  FewCounters* counters = reinterpret_cast<FewCounters*>(a.workspace + kStatusBytes);
  float* shares = reinterpret_cast<float*>(a.workspace + kStatusBytes + kCounterBytes);
  const size_t share = share_floats(a.tokens);
  uint16_t* act = reinterpret_cast<uint16_t*>(shares + 2 * kMaxCtas * share);

  // ---- setup: barriers, routing, the rows of every expert ----
  if (tid == 0) {
    for (int i = 0; i < sm.slots; ++i) {
      mbar_init(bar_w + 8 * i, 1);
      mbar_init(bar_x + 8 * i, 1);
      mbar_init(bar_e + 8 * i, 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
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
  for (int e = tid; e < a.num_experts; e += kFewThreads) s_mask[e] = 0u;
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
  uint32_t before = 0;  // rows | passes << 16 of the experts before mine
  uint32_t mine[2] = {0u, 0u};
  if (warp < kComputeWarps) {
    uint32_t own = 0;
    for (int i = 0; i < 2; ++i) {
      const int e = 2 * tid + i;
      mine[i] = e < a.num_experts ? s_mask[e] : 0u;
      const uint32_t n = __popc(mine[i]);
      own += n | ((n + kRowsPerPass - 1) / kRowsPerPass) << 16;
    }
    uint32_t incl = own;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    before = incl - own;
    if (lane == 31) warp_sums[warp] = static_cast<int>(incl);
  }
  __syncthreads();
  if (warp < kComputeWarps) {
    for (int i = 0; i < warp; ++i) before += static_cast<uint32_t>(warp_sums[i]);
    if (tid == kComputeThreads - 1) {
      uint32_t all = before;
      for (int i = 0; i < 2; ++i) {
        const uint32_t n = __popc(mine[i]);
        all += n | ((n + kRowsPerPass - 1) / kRowsPerPass) << 16;
      }
      *num_chunks_p = static_cast<int>(all >> 16);
    }
    for (int i = 0; i < 2; ++i) {
      const int e = 2 * tid + i;
      int row = static_cast<int>(before & 0xFFFFu), c = static_cast<int>(before >> 16);
      const int n = __popc(mine[i]);
      // expert | rows - 1 << 10 | first row << 16
      for (int r = 0; r < n; r += kRowsPerPass)
        chunks[c++] = static_cast<uint32_t>(e) |
                      static_cast<uint32_t>(min(kRowsPerPass, n - r) - 1) << 10 |
                      static_cast<uint32_t>(row + r) << 16;
      uint32_t m = mine[i];
      for (int r = 0; r < n; ++r) {
        const int t = __ffs(m) - 1;
        m &= m - 1;
        // the weight of an expert that a token names twice is the sum
        float w = 0.f;
        for (int s = 0; s < a.topk; ++s)
          if (s_ids[t * a.topk + s] == e) w += s_weights[t * a.topk + s];
        row_token[row + r] = t;
        row_weight[row + r] = w;
      }
      before += static_cast<uint32_t>(n) |
                static_cast<uint32_t>((n + kRowsPerPass - 1) / kRowsPerPass) << 16;
    }
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
  const int k_steps[2] = {(a.hidden + kKStep - 1) / kKStep, (a.inter + kKStep - 1) / kKStep};
  const int k_groups[2] = {a.hidden / kGroup, a.inter / kGroup};
  const int tiles[2] = {a.inter / 64, (a.hidden + kTileRows - 1) / kTileRows};
  Split split[2];
#pragma unroll
  for (int ph = 0; ph < 2; ++ph) {
    split[ph].stages = (k_steps[ph] + 1) / 2;
    split[ph].total = static_cast<long long>(num_chunks) * tiles[ph] * split[ph].stages;
    split[ph].grid = static_cast<int>(min(static_cast<long long>(gridDim.x), split[ph].total));
  }
  const int cta = blockIdx.x;

  if (warp == kComputeWarps) {
    // ---- weight copies (one thread) ----
    if (lane == 0) {
      const uint64_t policy = policy_evict_first();
      int slot = 0;
      uint32_t phase = 0;
      int issued = 0;
      bool ok = true;
#pragma unroll 1
      for (int ph = 0; ph < 2 && ok; ++ph) {
        if (cta >= split[ph].grid) continue;
        const long long begin = split[ph].begin(cta), end = split[ph].begin(cta + 1);
        const int S = split[ph].stages;
        long long q = begin / S;
        int s = static_cast<int>(begin - q * S);
        // gate_up: items by expert, then tile; down: by tile, then expert
        const int inner_n = ph == 0 ? tiles[0] : num_chunks;
        int outer = static_cast<int>(q / inner_n), inner = static_cast<int>(q % inner_n);
        const uint8_t* base = ph == 0 ? a.gate_up : a.down;
        const long long expert_bytes = ph == 0 ? a.gate_up_expert_bytes : a.down_expert_bytes;
        const uint8_t* src = nullptr;
        bool fresh = true;
        for (long long at = begin; at < end; ++at) {
          if (fresh) {
            const int c = ph == 0 ? outer : inner, tile = ph == 0 ? inner : outer;
            src = base + (chunks[c] & 1023u) * expert_bytes +
                  static_cast<long long>(tile) * k_steps[ph] * kStepBytes;
            fresh = false;
          }
          if (!few_wait(bar_e + 8 * slot, phase ^ 1u, abort_flag, status, kWhereRing,
                        a.timeout_cycles)) {
            ok = false;
            break;
          }
          const uint32_t bytes = min(2, k_steps[ph] - 2 * s) * kStepBytes;
          mbar_arrive_expect_tx(bar_w + 8 * slot, bytes);
          bulk_g2s(ring + slot * sm.slot_bytes, src + static_cast<long long>(s) * kWStage, bytes,
                   bar_w + 8 * slot, policy);
          ++issued;
          slot_next(slot, phase, 1, sm.slots);
          if (++s == S) {
            s = 0;
            fresh = true;
            if (++inner == inner_n) {
              inner = 0;
              ++outer;
            }
          }
        }
      }
      if (!ok)  // copies in flight land before the CTA ends
        for (int i = max(0, issued - sm.slots); i < issued; ++i) {
          const long long t0 = clock64();
          while (!mbar_try_wait(bar_w + 8 * (i % sm.slots), (i / sm.slots) & 1) &&
                 clock64() - t0 < kFewDrainCycles) {
          }
        }
    }
  } else if (warp == kComputeWarps + 1) {
    // ---- row copies: lane = part * 8 + row ----
    int slot = 0;
    uint32_t phase = 0;
    int issued = 0;
    bool ok = true;
    const int n8 = min(a.tokens, kRowsPerPass);
    const int r = lane & 7, part = lane >> 3;
#pragma unroll 1
    for (int ph = 0; ph < 2 && ok; ++ph) {
      if (cta >= split[ph].grid) continue;
      const long long begin = split[ph].begin(cta), end = split[ph].begin(cta + 1);
      const int S = split[ph].stages;
      const bool fp8 = kFp8 && ph == 0;
      const int parts = ph == 0 ? 1 : kParts;
      if (ph == 1) {
        // every gate_up item of every CTA is out
        bool seen = true;
        if (lane == 0) {
          const long long t0 = clock64();
          const int want = num_chunks * tiles[0];
          while (true) {
            int v;
            asm volatile("ld.acquire.gpu.global.b32 %0, [%1];"
                         : "=r"(v)
                         : "l"(&counters->act_done)
                         : "memory");
            if (v >= want) break;
            if (*abort_flag || clock64() - t0 > a.timeout_cycles) {
              if (!*abort_flag) atomicCAS(status, 0, 0x1000 | kWhereAct);
              *abort_flag = 1;
              seen = false;
              break;
            }
            __nanosleep(64);
          }
        }
        if (!__shfl_sync(0xffffffffu, seen, 0)) {
          ok = false;
          break;
        }
        __syncwarp();  // what lane 0 acquired is ordered before every lane's copies
        asm volatile("fence.proxy.async.global;" ::: "memory");
      }
      long long q = begin / S;
      int s = static_cast<int>(begin - q * S);
      const int inner_n = ph == 0 ? tiles[0] : num_chunks;
      int outer = static_cast<int>(q / inner_n), inner = static_cast<int>(q % inner_n);
      const uint8_t* src = nullptr;
      int n = 0;
      bool fresh = true;
      for (long long at = begin; at < end; ++at) {
        if (fresh) {
          const uint32_t ch = chunks[ph == 0 ? outer : inner];
          n = static_cast<int>((ch >> 10) & 7u) + 1;
          const int row = static_cast<int>(ch >> 16) + min(r, n - 1);
          if (ph == 0)
            src = static_cast<const uint8_t*>(a.x) +
                  static_cast<long long>(row_token[row]) * a.hidden * (fp8 ? 1 : 2);
          else
            src = reinterpret_cast<const uint8_t*>(act) +
                  (static_cast<long long>(row) * kParts + min(part, kParts - 1)) * a.inter * 2;
          fresh = false;
        }
        if (!__all_sync(0xffffffffu, few_wait(bar_e + 8 * slot, phase ^ 1u, abort_flag, status,
                                              kWhereRows, a.timeout_cycles))) {
          ok = false;
          break;
        }
        const uint32_t bytes =
            static_cast<uint32_t>(min(4, k_groups[ph] - 4 * s)) * (fp8 ? 32u : 64u);
        const uint32_t full = bar_x + 8 * slot;
        if (lane == 0) mbar_arrive_expect_tx(full, bytes * n * parts);
        __syncwarp();
        if (r < n && part < parts) {
          const uint32_t dst = ring + slot * sm.slot_bytes + kWStage +
                               (fp8 ? r * kRowPitchFp8 : (part * n8 + r) * kRowPitch);
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
              "[%0], [%1], %2, [%3];" ::"r"(dst),
              "l"(src + static_cast<long long>(s) * (fp8 ? kStageK : 2 * kStageK)), "r"(bytes),
              "r"(full)
              : "memory");
        }
        ++issued;
        slot_next(slot, phase, 1, sm.slots);
        if (++s == S) {
          s = 0;
          fresh = true;
          if (++inner == inner_n) {
            inner = 0;
            ++outer;
          }
        }
      }
    }
    if (!ok && lane == 0)
      for (int i = max(0, issued - sm.slots); i < issued; ++i) {
        const long long t0 = clock64();
        while (!mbar_try_wait(bar_x + 8 * (i % sm.slots), (i / sm.slots) & 1) &&
               clock64() - t0 < kFewDrainCycles) {
        }
      }
  } else {
    // ---- compute: warpgroup `grp` takes the stages u % 4 == grp ----
    // After a wait gave up every warp still walks its stages (on whatever the
    // ring holds), so that all barriers among the compute warps are met.
    const int grp = warp >> 2;
    const int m0 = (warp & 3) * 32;  // this warp's weight rows in a tile
    const int g = lane >> 2, t = lane & 3;
    int slot = grp;                  // slot and phase of this group's next stage
    uint32_t phase = 0;
    int u = 0;                       // stages of this CTA before the current segment
    bool live = true;
    const int n8 = min(a.tokens, kRowsPerPass);
    const uint32_t part_bytes = n8 * kRowPitch;
    const int x_groups = split[0].stages;

#pragma unroll 1
    for (int ph = 0; ph < 2; ++ph) {
      if (cta >= split[ph].grid) continue;
      const long long begin = split[ph].begin(cta), end = split[ph].begin(cta + 1);
      const int S = split[ph].stages;
      const int inner_n = ph == 0 ? tiles[0] : num_chunks;
      long long q = begin / S;
      int s0 = static_cast<int>(begin - q * S);
      int outer = static_cast<int>(q / inner_n), inner = static_cast<int>(q % inner_n);
      long long at = begin;
      if (ph == 1) {
        for (int i = tid; i < kGroups * max(a.tokens, kRowsPerPass) * kSumPitch;
             i += kComputeThreads)
          sums[i] = 0.f;
        compute_sync();
      }
      while (at < end) {
        const int len = static_cast<int>(min(static_cast<long long>(S - s0), end - at));
        const uint32_t ch = chunks[ph == 0 ? outer : inner];
        const int n = static_cast<int>((ch >> 10) & 7u) + 1;
        const int row0 = static_cast<int>(ch >> 16);
        const int first = s0 + ((grp - u) & 3);
        float acc[2][4] = {};
        const uint32_t col = g < n ? g : 0;  // columns past the rows repeat row 0, unused
        const uint32_t row_at =
            kWStage + (kFp8 && ph == 0 ? col * kRowPitchFp8 + t * 8 : col * kRowPitch + t * 16);
        const uint32_t codes_at = (m0 + lane) * 16;
        const uint32_t scales_at = kStepQBytes + (m0 + g) * 2;
#pragma unroll 1
        for (int s = first; s < s0 + len; s += kGroups) {
          if (live)
            live = __all_sync(0xffffffffu,
                              few_wait(bar_w + 8 * slot, phase, abort_flag, status, kWhereData,
                                       a.timeout_cycles) &&
                                  few_wait(bar_x + 8 * slot, phase, abort_flag, status,
                                           kWhereData, a.timeout_cycles));
          const uint32_t base = ring + slot * sm.slot_bytes;
          const int valid = min(4, k_groups[ph] - 4 * s);
          if (ph == 0) {
            if constexpr (kFp8) {
              // the rows' scales cover exactly one stage
              float part[2][4] = {};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (i < valid)
                  group_mma<1, true>(base + (i >> 1) * kStepBytes + (i & 1) * 2048 + codes_at,
                                     base + (i >> 1) * kStepBytes + (i & 1) * 256 + scales_at,
                                     base + row_at + i * 32, 0, part);
              const int c0 = min(2 * t, n - 1), c1 = min(2 * t + 1, n - 1);
              const float x0 = s_xscales[row_token[row0 + c0] * x_groups + s];
              const float x1 = s_xscales[row_token[row0 + c1] * x_groups + s];
#pragma unroll
              for (int mt = 0; mt < 2; ++mt) {
                acc[mt][0] = fmaf(x0, part[mt][0], acc[mt][0]);
                acc[mt][1] = fmaf(x1, part[mt][1], acc[mt][1]);
                acc[mt][2] = fmaf(x0, part[mt][2], acc[mt][2]);
                acc[mt][3] = fmaf(x1, part[mt][3], acc[mt][3]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (i < valid)
                  group_mma<1, false>(base + (i >> 1) * kStepBytes + (i & 1) * 2048 + codes_at,
                                      base + (i >> 1) * kStepBytes + (i & 1) * 256 + scales_at,
                                      base + row_at + i * 64, 0, acc);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i < valid)
                group_mma<kParts, false>(base + (i >> 1) * kStepBytes + (i & 1) * 2048 + codes_at,
                                         base + (i >> 1) * kStepBytes + (i & 1) * 256 + scales_at,
                                         base + row_at + i * 64, part_bytes, acc);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_e + 8 * slot);
          slot_next(slot, phase, kGroups, sm.slots);
        }
        at += len;
        u += len;
        const bool item_end = s0 + len == S;
        float* my = sums + grp * max(a.tokens, kRowsPerPass) * kSumPitch;

        if (ph == 0) {
          // the item's share of this CTA: [row of the pass][128], four groups
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              my[(2 * t + (i & 1)) * kSumPitch + m0 + mt * 16 + (i >> 1) * 8 + g] = acc[mt][i];
          compute_sync();
          const int stride = max(a.tokens, kRowsPerPass) * kSumPitch;
          const bool whole = s0 == 0 && item_end;
          bool finish = whole;
          const long long item0 = (static_cast<long long>(outer) * inner_n + inner) * S;
          const int cta0 = split[0].owner(item0), cta1 = split[0].owner(item0 + S - 1);
          if (!whole) {
            // a share goes out; the CTA that arrives last adds them all
            float* dst = shares + (2 * cta + (cta == cta0 ? 1 : 0)) * share;
            for (int i = tid; i < n * kTileRows; i += kComputeThreads) {
              const float* from = sums + (i >> 7) * kSumPitch + (i & 127);
              __stcg(dst + i, (from[0] + from[stride]) + (from[2 * stride] + from[3 * stride]));
            }
            __threadfence();
            compute_sync();
            if (tid == 0) {
              *last_arrival = atomicAdd(&counters->item[0][cta0], 1) == cta1 - cta0;
              __threadfence();
            }
            compute_sync();
            finish = *last_arrival != 0;
          }
          if (finish) {
            // act = silu(gate) * up of 64 columns x n rows, as three BF16 parts
            for (int i = tid; i < n * 64; i += kComputeThreads) {
              const int c = i & 63, r = i >> 6;
              const int at_g = (c >> 4) * 32 + (c & 15);
              float gate, up;
              if (whole) {
                const float* from = sums + r * kSumPitch + at_g;
                gate = (from[0] + from[stride]) + (from[2 * stride] + from[3 * stride]);
                from += 16;
                up = (from[0] + from[stride]) + (from[2 * stride] + from[3 * stride]);
              } else {
                gate = up = 0.f;
                for (int b = cta0; b <= cta1; ++b) {
                  const float* from =
                      shares + (2 * b + (b == cta0 ? 1 : 0)) * share + r * kTileRows + at_g;
                  gate += __ldcg(from);
                  up += __ldcg(from + 16);
                }
              }
              const float v = gate / (1.f + expf(-gate)) * up;
              uint16_t* dst = act + (static_cast<long long>(row0 + r) * kParts) * a.inter +
                              inner * 64 + c;
              const uint32_t bits = __float_as_uint(v);
              if ((bits & 0x7F800000u) == 0x7F800000u) {  // infinity or NaN: one part
                dst[0] = static_cast<uint16_t>(bits >> 16) | ((bits & 0xFFFFu) != 0 ? 0x40 : 0);
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
            }
            __threadfence();
          }
          compute_sync();  // the sums are free again; every part is out
          if (finish && tid == 0) {
            __threadfence();
            atomicAdd(&counters->act_done, 1);
          }
        } else {
          // this group's share of the tile: the pass's rows at their tokens
          if (first < s0 + len) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int c = 2 * t + i;
              if (c < n) {
                const float w = row_weight[row0 + c];
                float* dst = my + row_token[row0 + c] * kSumPitch + m0 + g;
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                  dst[mt * 16] = fmaf(w, acc[mt][i], dst[mt * 16]);
                  dst[mt * 16 + 8] = fmaf(w, acc[mt][2 + i], dst[mt * 16 + 8]);
                }
              }
            }
            __syncwarp();
          }
          const bool tile_end = item_end && inner + 1 == inner_n;
          if (tile_end || at == end) {
            const int tile = outer;
            const long long tile0 = static_cast<long long>(tile) * inner_n * S;
            const int cta0 = split[1].owner(tile0),
                      cta1 = split[1].owner(tile0 + static_cast<long long>(inner_n) * S - 1);
            const int stride = max(a.tokens, kRowsPerPass) * kSumPitch;
            const int h0 = tile * kTileRows;
            compute_sync();
            float* dst = shares + (2 * cta + (cta == cta0 ? 1 : 0)) * share;
            for (int i = tid; i < a.tokens * kTileRows; i += kComputeThreads) {
              const int tok = i >> 7, h = i & 127;
              float* from = sums + tok * kSumPitch + h;
              const float v = (from[0] + from[stride]) + (from[2 * stride] + from[3 * stride]);
              from[0] = from[stride] = from[2 * stride] = from[3 * stride] = 0.f;
              if (cta0 != cta1) {
                __stcg(dst + i, v);
              } else if (h0 + h < a.hidden) {
                float* o = a.out + static_cast<long long>(tok) * a.hidden + h0 + h;
                *o = a.accumulate ? *o + v : v;
              }
            }
            if (cta0 != cta1) {
              __threadfence();
              compute_sync();
              if (tid == 0) {
                *last_arrival = atomicAdd(&counters->item[1][cta0], 1) == cta1 - cta0;
                __threadfence();
              }
              compute_sync();
              if (*last_arrival) {
                for (int i = tid; i < a.tokens * kTileRows; i += kComputeThreads) {
                  const int tok = i >> 7, h = i & 127;
                  if (h0 + h >= a.hidden) continue;
                  float v = 0.f;
                  for (int b = cta0; b <= cta1; ++b)
                    v += __ldcg(shares + (2 * b + (b == cta0 ? 1 : 0)) * share + i);
                  float* o = a.out + static_cast<long long>(tok) * a.hidden + h0 + h;
                  *o = a.accumulate ? *o + v : v;
                }
              }
            }
            compute_sync();
          }
        }
        s0 = 0;
        if (++inner == inner_n) {
          inner = 0;
          ++outer;
        }
      }
    }
    // the last CTA out leaves the counters zero for the next call
    compute_sync();
    if (tid == 0) {
      __threadfence();
      *last_arrival = atomicAdd(&counters->exits, 1) == static_cast<int>(gridDim.x) - 1;
    }
    compute_sync();
    if (*last_arrival) {
      for (int i = tid; i < 2 * kMaxCtas; i += kComputeThreads) counters->item[0][i] = 0;
      if (tid == 0) {
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
