// product_few.cu -- products with one weight, packed INT4 or BF16, for up to 32
// tokens (but INT4 ones of many rows for more than 16), plain or gated:
//
//   out[t, r] = addend[t, r] + x[t] . w[r]^T
//   out[t, i] = silu(x[t] . wgate[i]^T) * (x[t] . wup[i]^T)
//
// The weight is the traffic, and the time is that of reading it once, plus a
// launch, a first load and the sums' way out. Every warp copies its own steps of
// 64 columns into slots of its own (no barrier between warps before the sums),
// several steps ahead, and multiplies with m16n8k16 MMAs whose M side are the
// weight rows. The packed codes become BF16 numbers q - 8, and a group's scale is
// applied to its FP32 sum, so no weight is rounded.
//
// One token, in a graph: BF16, 4096 x 7168 gated 10.0 us, 5.9 TB/s (0.86 of the
// copy rate); INT4, the same 5.7 us for 16.5 MB, 7168 x 2048 4.0 us, where launch,
// first load and sums are some 3 us; 16384 x 7168 15.2 us, 4.3 TB/s: the ALU pipe
// (a shift and an AND-OR for two codes, at half rate) is busy two thirds of the
// time, and 256 blocks on 152 SMs leave a sixth of it out.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "product_out.cuh"
#include "ptx.cuh"

namespace w4a16 {

namespace {

// d = a . b + c, BF16 operands
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
        "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
}

// Rows of 128 bytes, 16-byte chunks c of odd rows in the other half, so that the
// eight lanes of two rows that load at a time meet all banks.
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
  return static_cast<uint32_t>(row * 128 + ((c ^ (row & 1) << 2) << 4));
}

struct FewProduct {
  ProductArgs a;
  int blocks;         // of a cluster's rows
  int split;          // CTAs of a cluster, which share the columns
  int steps;          // of 64 columns
  int slot_bytes;     // of a warp's step
  uint32_t sixteens;  // 16 as two BF16 numbers
};

// Bytes of a step of 64 columns of a warp's rows and of the tokens.
constexpr int step_bytes(bool int4, int rows) { return rows * (int4 ? 36 : 128); }

}  // namespace

// A cluster has blocks of 16 * kMt weight rows, one after the other, a CTA of it a
// share of their columns, of which its warps take steps of 64 by turns. A warp
// copies its steps (the weights, and the tokens' columns) into slots of its own,
// kDepth ahead and on into the next block. The sums of the warps meet in shared
// memory, those of the CTAs through the cluster's.
template <bool kInt4, bool kGated, int kMt, int kNt, int kDepth, int kWarps>
__global__ void __launch_bounds__(kWarps * 32) w4a16_product_few_kernel(const FewProduct p) {
  constexpr int kThreads = kWarps * 32;
  constexpr int kRows = 16 * kMt;
  constexpr int kTokens = 8 * kNt;
  constexpr int kPitch = kRows + kSumPad;  // of a token's sums
  static_assert(kMt % 2 == 0, "gate and up rows by sixteens, codes by 32 rows");
  extern __shared__ __align__(128) uint8_t smem[];
  const ProductArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int begin = static_cast<int>(blockIdx.x) / p.split;
  const int stride = static_cast<int>(gridDim.x) / p.split;
  const int columns = kGated ? a.n / 2 : a.n;
  const int first = p.steps * rank / p.split + warp, last = p.steps * (rank + 1) / p.split;
  const uint32_t slots = smem_u32(smem) + static_cast<uint32_t>(warp * kDepth * p.slot_bytes);
  // [kWarps / 2][kTokens][kPitch]
  float* part = reinterpret_cast<float*>(smem + kWarps * kDepth * p.slot_bytes);
  constexpr uint32_t kWeightBytes = step_bytes(kInt4, kRows);
  // This lane's sources in the step that it fetches next. (k is a multiple of 8,
  // and a packed step is whole: only chunks of x, and of BF16 weights, can lie
  // behind the row's end.)
  constexpr int kWeightCopies = kInt4 ? kRows / 16 : kRows / 4;
  const uint8_t* w_from[kInt4 ? 2 : kWeightCopies];
  const uint16_t* x_from;
  int c_from, next_block = first < last ? begin : p.blocks, next_step;
  const auto point = [&](int block) {
    if constexpr (kInt4) {
      const int r0 = block * kRows;
      const uint8_t* from = static_cast<const uint8_t*>(a.weight) +
                            (static_cast<long long>(r0 / kTileRows) * p.steps + first) * kStepBytes;
      w_from[0] = from + (r0 % kTileRows + lane) * 16;  // codes of row `lane`
      w_from[1] = from + kStepQBytes + lane / (kRows / 8) * (kTileRows * 2) + r0 % kTileRows * 2 +
                  lane % (kRows / 8) * 16;
    } else {
#pragma unroll
      for (int j = 0; j < kWeightCopies; ++j) {
        const int r = 4 * j + (lane >> 3);
        int q = min(block * kRows + r, columns - 1);  // weight row
        if constexpr (kGated)
          q = min(block * (kRows / 2) + r / 32 * 16 + r % 16, columns - 1) + r / 16 % 2 * columns;
        w_from[j] = static_cast<const uint8_t*>(a.weight) +
                    (static_cast<long long>(q) * a.k + first * kKStep + (lane & 7) * 8) * 2;
      }
    }
    next_step = first;
    c_from = first * kKStep + (lane & 7) * 8;
    x_from = a.x + min(lane >> 3, a.tokens - 1) * a.x_stride + c_from;
  };
  point(begin);
  // The weights of the first steps set out while the kernel before is still at work
  // (one after another, one token: BF16 4096 x 7168 10.5 -> 10.0 us, 7168 x 2048 6.6 ->
  // 5.9; INT4 6.1 -> 5.9, 4.4 -> 4.0, 16384 x 7168 16.3 -> 15.2).
  if (first < last && begin < p.blocks) {
#pragma unroll 1
    for (int d = 0; d < kDepth && first + d * kWarps < last; ++d) {
      if constexpr (kInt4) {
#pragma unroll
        for (int j = 0; j < kWeightCopies; ++j)
          prefetch_l2(w_from[0] + static_cast<long long>(d) * kWarps * kStepBytes +
                      j / (kRows / 32) * (kTileRows * 16) + j % (kRows / 32) * 512);
        if (lane < kRows / 4)
          prefetch_l2(w_from[1] + static_cast<long long>(d) * kWarps * kStepBytes);
      } else {
#pragma unroll
        for (int j = 0; j < kWeightCopies; ++j)
          if (c_from + d * kWarps * kKStep < a.k) prefetch_l2(w_from[j] + d * kWarps * kKStep * 2);
      }
    }
  }
  grid_dependency_wait();
  grid_dependents_go();

  const uint32_t x_to = kWeightBytes + chunk_at(lane >> 3, lane & 7), w_to = lane * 16;
  const long long x_four = 4 * a.x_stride;
  const int x_last = a.tokens - 1 - (lane >> 3);
  const auto fetch = [&](uint32_t slot) {
    if (next_block >= p.blocks) return;
    const int bytes = c_from < a.k ? 16 : 0;
    if constexpr (kInt4) {
#pragma unroll
      for (int j = 0; j < kWeightCopies; ++j)  // codes [half][row][16]
        copy16(slot + w_to + j * 512,
               w_from[0] + j / (kRows / 32) * (kTileRows * 16) + j % (kRows / 32) * 512);
      if (lane < kRows / 4)  // scales [half][row]
        copy16(slot + w_to + 2 * kRows * 16, w_from[1]);
      w_from[0] += kWarps * kStepBytes;
      w_from[1] += kWarps * kStepBytes;
    } else {
#pragma unroll
      for (int j = 0; j < kWeightCopies; ++j) {
        copy16_of(slot + x_to - kWeightBytes + j * 512, w_from[j], bytes);
        w_from[j] += kWarps * kKStep * 2;
      }
    }
    const uint16_t* from = x_from;
#pragma unroll
    for (int j = 0; j < 2 * kNt; ++j, from += x_four)
      if (4 * j <= x_last) copy16_of(slot + x_to + j * 512, from, bytes);
    x_from += kWarps * kKStep;
    c_from += kWarps * kKStep;
    next_step += kWarps;
    if (next_step >= last) {
      next_block += stride;
      if (next_block < p.blocks) point(next_block);
    }
  };

  float acc[kMt][kNt][4];
  uint32_t x_row[kNt][2];
#pragma unroll
  for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      x_row[nt][h] = kWeightBytes + chunk_at(min(8 * nt + g, a.tokens - 1), 4 * h + t);
  const auto multiply = [&](uint32_t slot) {
    uint32_t sc[kMt / 2][4];
    if constexpr (kInt4) {
      // lane = (matrix, row): matrix m gives rows 16 (m & 1) .. + 15 of half
      // m >> 1; its eight addresses alternate between rows + 0 and rows + 8
      const uint32_t scales = slot + 2 * kRows * 16 + (lane >> 4) * (kRows * 2) +
                              ((lane >> 3 & 1) * 16 + (lane & 1) * 8) * 2;
#pragma unroll
      for (int j = 0; j < kMt / 2; ++j) ldmatrix_x4_trans(scales + j * 64, sc[j]);
    }
    uint4 x[2][kNt];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) x[h][nt] = load_shared16(slot + x_row[nt][h]);
    const float none[4] = {};
    if constexpr (kInt4) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < kMt / 2; ++j) {
          uint32_t w[4];
          ldmatrix_x4(slot + (h * kRows + j * 32 + lane) * 16, w);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int mt = 2 * j + i;
            const uint32_t w0 = w[2 * i], w1 = w[2 * i + 1];
            const auto code = [&](uint32_t v) { return code_pair(v, p.sixteens); };
            const uint32_t a0[4] = {code(w0 << 3), code(w1 << 3), code(w0 >> 1), code(w1 >> 1)};
            const uint32_t a1[4] = {code(w0 >> 5), code(w1 >> 5), code(w0 >> 9), code(w1 >> 9)};
            const uint32_t pair = sc[j][2 * h + i];
            const float s0 = __uint_as_float(pair << 16), s1 = __uint_as_float(pair & 0xFFFF0000u);
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) {
              float c[4];
              mma16816(c, a0, x[h][nt].x, x[h][nt].y, none);
              mma16816(c, a1, x[h][nt].z, x[h][nt].w, c);
              fma_pair(acc[mt][nt][0], acc[mt][nt][1], s0, c[0], c[1]);
              fma_pair(acc[mt][nt][2], acc[mt][nt][3], s1, c[2], c[3]);
            }
          }
        }
    } else {
      // (a step's sum of its own: the tensor core cuts off at every addition, over a
      // warp's share of 7168 columns 8.6e-7 of the result)
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
        uint32_t w[2][2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t at = slot + mt * 2048 + chunk_at(g, 4 * h + t);
          const uint4 w0 = load_shared16(at), w1 = load_shared16(at + 8 * 128);
          const uint32_t a0[4] = {w0.x, w1.x, w0.y, w1.y}, a1[4] = {w0.z, w1.z, w0.w, w1.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) w[h][0][i] = a0[i], w[h][1][i] = a1[i];
        }
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) {
          float c[4];
          mma16816(c, w[0][0], x[0][nt].x, x[0][nt].y, none);
          mma16816(c, w[0][1], x[0][nt].z, x[0][nt].w, c);
          mma16816(c, w[1][0], x[1][nt].x, x[1][nt].y, c);
          mma16816(c, w[1][1], x[1][nt].z, x[1][nt].w, c);
          fma_pair(acc[mt][nt][0], acc[mt][nt][1], 1.f, c[0], c[1]);
          fma_pair(acc[mt][nt][2], acc[mt][nt][3], 1.f, c[2], c[3]);
        }
      }
    }
  };

  // a group of copies a slot, also an empty one
#pragma unroll 1
  for (int d = 0; d < kDepth; ++d) {
    fetch(slots + d * p.slot_bytes);
    copies_commit();
  }
  uint32_t slot = slots;
#pragma unroll 1
  for (int block = begin; block < p.blocks; block += stride) {
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;
#pragma unroll 1
    for (int step = first; step < last; step += kWarps) {
      copies_wait<kDepth - 1>();
      __syncwarp();
      multiply(slot);
      __syncwarp();
      fetch(slot);
      copies_commit();
      slot += p.slot_bytes;
      if (slot == slots + kDepth * p.slot_bytes) slot = slots;
    }
    // the sums of the upper half of the warps, on to those of the lower half
    const auto each = [&](auto use) {
      float* mine = part + ((warp % (kWarps / 2)) * kTokens + 2 * t) * kPitch + g;
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            use(mine[(8 * nt + (i & 1)) * kPitch + mt * 16 + (i >> 1) * 8], acc[mt][nt][i]);
    };
    __syncthreads();  // the block before is out
    if (warp >= kWarps / 2) each([](float& at, float v) { at = v; });
    __syncthreads();
    if (warp < kWarps / 2) each([](float& at, float v) { at += v; });
    __syncthreads();
    for (int i = threadIdx.x; i < a.tokens * kRows; i += kThreads) {
      const int at = i / kRows * kPitch + i % kRows;
      float v = part[at];
#pragma unroll
      for (int s = 1; s < kWarps / 2; ++s) v += part[s * kTokens * kPitch + at];
      part[at] = v;
    }
    if (p.split > 1)
      cluster_sync_all();
    else
      __syncthreads();
    // every CTA of the cluster writes its share of the outputs
    write_products<kGated, kRows>(a, part, block, rank * kThreads + static_cast<int>(threadIdx.x),
                                  p.split * kThreads, p.split);
    if (p.split > 1) cluster_sync_all();  // the sums stay until all have read them
  }
}

namespace {

template <bool kInt4, bool kGated, int kMt, int kNt, int kDepth, int kWarps = 8>
cudaError_t run(const ProductArgs& args, int sms, cudaStream_t stream) {
  constexpr int kRows = 16 * kMt;
  const auto kernel = w4a16_product_few_kernel<kInt4, kGated, kMt, kNt, kDepth, kWarps>;
  FewProduct p;
  p.a = args;
  p.sixteens = 0x41804180u;
  p.blocks = ceil_div(args.n, kRows);
  p.steps = ceil_div(args.k, kKStep);
  p.slot_bytes = step_bytes(kInt4, kRows) + args.tokens * 128;
  // a cluster of two, four or eight where all CTAs still find an SM and every warp a
  // step; eights, which do not all find a place at once, on half of the SMs. (One
  // token and 7168 columns, BF16: 128 rows in eights 2.7 us, in fours 3.3; 32 tokens
  // and 512 rows, INT4: 8.2 in eights, 4.9 in fours.)
  p.split = 1;
  while (p.split < 8 && (p.split < 4 ? 2 : 4) * p.blocks * p.split <= sms &&
         p.steps >= 2 * p.split * kWarps)
    p.split *= 2;
  // Where every CTA has an SM of its own, no two of them may share one: those of the
  // next launch, which come early, would crowd into the SMs that this one leaves out
  // (launches one after another of 4096 x 7168, INT4, one token: 6.2 -> 5.7 us).
  int smem = kWarps * kDepth * p.slot_bytes + kWarps / 2 * 8 * kNt * (kRows + kSumPad) * 4;
  if (p.blocks <= sms) smem = std::max(smem, kMaxSmem / 2 + 1);
  if (smem > 48 << 10) {
    static Devices known{0};
    const cudaError_t e = allow_smem(kernel, kMaxSmem, known);
    if (e != cudaSuccess) return e;
  }
  // as many CTAs as the SMs hold
  const int an_sm = std::min(4, kMaxSmem / smem);
  const int clusters = p.split > 1 ? p.blocks : std::min(p.blocks, an_sm * sms);
  return launch_dependent(kernel, clusters * p.split, kWarps * 32, static_cast<size_t>(smem),
                          p.split, stream, p);
}

}  // namespace

// Rows of a block and steps in flight by the tokens, and by whether blocks of 32
// rows are at most one an SM (us in a graph, weights not in L2, hidden 7168 unless
// said):
//   INT4, one token, 9728 rows: 32 x 5 10.4, 64 x 4 10.0; 16384 rows 17.9, 15.4; 7168 x
//     2048 4.1, 4.2; 4096 rows 6.5, 7.1, and with 16 warps for eight 32 x 3 5.8 (1024
//     rows: 4.1 with either)
//   INT4, 16 tokens, 9728 rows: 32 x 4 12.8, 64 x 5 12.9; 16384 rows 23.2, 22.7; 4096
//     rows 7.4, 8.4
//   INT4, 32 tokens, 4096 rows: 32 x 2 10.3, 32 x 3 10.0, 64 x 3 11.7; 9728 rows 20.6,
//     19.7, 17.5; 7168 x 2048 9.1, 8.3, 7.4
//   BF16, one token, 4096 rows: 32 x 5 10.7, 32 x 3 11.1; 7168 x 2048 6.2, 6.2; 18432
//     rows 40.2, 40.9
//   BF16, 16 tokens, 4096 rows: 32 x 4 11.5, 32 x 2 12.8; 7168 x 2048 7.1, 7.0
//   BF16, 32 tokens, 4096 rows: 32 x 3 13.0, 64 x 2 15.4; 7168 x 2048 9.9, 9.5; 18432
//     rows 47.5, 47.9
// INT4 rows more than 64 an SM and more than 16 tokens go to tcgen05 (us of mma.sync
// and of tcgen05, 32 tokens; with 17 both are 3 % faster): 12288 rows 28.7 to 32.1, 23.1;
// 16384 32.6, 23.4; 32768 63.6, 45.1; 16384 x 2048 13.4, 10.2. With fewer rows blocks
// of 128 are on half of the SMs or fewer, and a block takes what it takes: 9728 rows
// 17.5, 23.0, 9728 x 2048 8.0, 9.3, and 4096 rows 10.0, 22.6. 16 tokens are half of the
// MMAs: 16384 rows 22.7, 20.9, but 65536 74.6, 75.9.
template <bool kInt4, bool kGated>
cudaError_t few(const ProductArgs& args, int sms, cudaStream_t stream) {
  const bool one = args.n <= 32 * sms;
  if constexpr (kInt4) {
    if (args.tokens <= 8 && one && args.n > 16 * sms)  // (no cluster either)
      return run<kInt4, kGated, 2, 1, 3, 16>(args, sms, stream);
    if (args.tokens <= 8)
      return one ? run<kInt4, kGated, 2, 1, 5>(args, sms, stream)
                 : run<kInt4, kGated, 4, 1, 4>(args, sms, stream);
    if (args.tokens <= 16)
      return one ? run<kInt4, kGated, 2, 2, 4>(args, sms, stream)
                 : run<kInt4, kGated, 4, 2, 5>(args, sms, stream);
    if (args.n > 64 * sms) return launch_linear_tmem(args, sms, stream);
    return one ? run<kInt4, kGated, 2, 4, 3>(args, sms, stream)
               : run<kInt4, kGated, 4, 4, 3>(args, sms, stream);
  } else {
    if (args.tokens <= 8)
      return one ? run<kInt4, kGated, 2, 1, 5>(args, sms, stream)
                 : run<kInt4, kGated, 2, 1, 3>(args, sms, stream);
    if (args.tokens <= 16)
      return one ? run<kInt4, kGated, 2, 2, 4>(args, sms, stream)
                 : run<kInt4, kGated, 2, 2, 2>(args, sms, stream);
    return one ? run<kInt4, kGated, 2, 4, 3>(args, sms, stream)
               : run<kInt4, kGated, 4, 4, 2>(args, sms, stream);
  }
}

cudaError_t launch_linear_few(const ProductArgs& args, int sms, cudaStream_t stream) {
  return args.gated ? few<true, true>(args, sms, stream) : few<true, false>(args, sms, stream);
}

cudaError_t launch_dense_few(const ProductArgs& args, int sms, cudaStream_t stream) {
  return args.gated ? few<false, true>(args, sms, stream) : few<false, false>(args, sms, stream);
}

}  // namespace w4a16
