// dense.cu -- products with one BF16 weight for many tokens, plain or gated:
//
//   out[t, r] = addend[t, r] + x[t] . w[r]^T
//   out[t, i] = silu(x[t] . wgate[i]^T) * (x[t] . wup[i]^T)
//
// tcgen05 with 256 tokens x up to 256 weight rows a tile, by pairs of CTAs that go
// from tile to tile; or, where there are fewer tiles than SMs, 128 tokens a tile
// with the columns split over a cluster. A gated tile has as many gate as up
// rows, so a token's gate and up lie in one TMEM lane.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "pipe.cuh"
#include "ptx.cuh"
#include "silu.cuh"

namespace w4a16 {

namespace {

constexpr int kTileM = 128;      // tokens of a CTA
constexpr int kSumWarps = 8;     // two a TMEM quarter, half of the columns each
constexpr int kWarpCopy = kSumWarps, kWarpMma = kSumWarps + 1;
constexpr int kDenseThreads = 32 * (kSumWarps + 4);  // whole warpgroups: two warps do nothing
constexpr int kMaxSlots = 8;
// The tensor core cuts its running sums off instead of rounding them: 1.5e-6 of an
// FP32 output after the 128 additions that 2048 columns are, and more with every
// column. So an accumulator's sums go to FP32 sums in registers, for FP32 outputs
// after 512 columns: 3.4e-7 (a plain FP32 product: 2.8e-7), for 169 instead of 146 us
// of 8192 x 2048 x 7168; after 256 columns 1.7e-7 and 183 us. For BF16 outputs, which
// it moves over a border now and then, after 1024: 576 tokens of 4096 x 7168 gated
// are 2.9e-4 off the rounded 64-bit result with one accumulator, 1.2e-4 with 2048
// columns, 0.9e-4 with 1024 and 0.6e-4 with 512, which take 36.6, 36.6, 36.6 and 36.8
// us; 8192 x 2048 x 7168 150, 150, 150 and 170.
constexpr int kRun = 8, kRunRounded = 16;
constexpr int kChunk = 32;       // output columns of an epilogue warp at a time
constexpr int kTileBytes = 32 * kChunk * 4;  // of its 32 tokens
constexpr int kTilesBytes = kSumWarps * 2 * kTileBytes;
constexpr int kRingBytes = 160 << 10;
constexpr int kSmemBytes = 1024 + kRingBytes + kTilesBytes;

// The tokens that a CTA multiplies when it has those from m0 on: 128 whole ones,
// the last 128 where fewer (or none) are left. It writes only its own. (Rows that
// the copy would fill with zeros behind the last token make the MMAs slower: a
// tile of 255 tokens took 48 us, one of 256 41, one of 256 zero tokens 48.)
__device__ __forceinline__ int first_token(int m0, int tokens) {
  return max(min(m0, tokens - kTileM), 0);
}

struct DenseArgs {
  CUtensorMap x, weight;
  ProductArgs a;
  int columns;       // of the output
  int half;          // weight rows of a box: half of a tile's
  int out_cols;      // output columns of a tile
  int m_tiles, n_tiles, k_steps;
  int slots;
  int run;           // steps of an accumulator before its sums are added in registers
  int split;         // CTAs of a cluster that share a tile's columns of x (split kernel)
  long long wait_limit;  // cycles
};

// The sums of a lane: kGroups groups of 16 columns, group g those from the
// accumulator's column at(g) on, taken over (fresh) or added. Groups from `used` on
// are left out (none where it is kGroups). One group at a time: more in flight are
// no faster and need registers.
constexpr int kGroups = 8;
template <typename At>
__device__ __forceinline__ void take_sums(float (&sum)[kGroups][16], bool fresh, int used, At at) {
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    if (g >= used) break;
    uint32_t v[16];
    tmem_ld_32x32b_x16(at(g), v);
    tmem_ld_wait_for(v);
#pragma unroll
    for (int c = 0; c < 16; ++c)
      sum[g][c] = __uint_as_float(v[c]) + (fresh ? 0.f : sum[g][c]);
  }
}

// Offset of four columns of a row in a warp's tile of 32 x 32 floats, placed so
// that both a column of rows and a row meet all banks.
__device__ __forceinline__ int tile_at(int row, int quad) {
  return row * kChunk + ((quad ^ (row & 7)) << 2);
}

// Four adjacent output values of a token, the columns from c on.
__device__ __forceinline__ float4 load_addend(const DenseArgs& p, int token, int c) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.a.addend == nullptr || token >= p.a.tokens || c >= p.columns) return v;
  const float* at = p.a.addend + static_cast<long long>(token) * p.columns + c;
  if (p.columns % 4 == 0) return *reinterpret_cast<const float4*>(at);
  float f[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c + i < p.columns) f[i] = at[i];
  return make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ uint2 bf16x4(float4 v) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                    *reinterpret_cast<const uint32_t*>(&hi));
}
__device__ __forceinline__ void store_out(const DenseArgs& p, int token, int c, float4 v) {
  if (token >= p.a.tokens || c >= p.columns) return;
  const long long at = static_cast<long long>(token) * p.columns + c;
  const float f[4] = {v.x, v.y, v.z, v.w};
  if (p.a.f32_out) {
    float* out = static_cast<float*>(p.a.out) + at;
    if (p.columns % 4 == 0) {
      *reinterpret_cast<float4*>(out) = v;
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < p.columns) out[i] = f[i];
  } else {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.out) + at;
    if (p.columns % 4 == 0) {
      *reinterpret_cast<uint2*>(out) = bf16x4(v);
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < p.columns) out[i] = __float2bfloat16_rn(f[i]);
  }
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

}  // namespace

// Pairs of CTAs: each copies its own 128 tokens and half of the tile's weight
// rows (gated: one the gate rows, the other the up rows), the first CTA's MMA
// thread issues for both, and every CTA keeps the sums of its tokens. Two
// accumulators, so that a tile's sums leave while the next one is multiplied.
__global__ void __launch_bounds__(kDenseThreads, 1)
    w4a16_dense_pair_kernel(const __grid_constant__ DenseArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t bars[2 * kMaxSlots + 5];
  __shared__ uint32_t tmem_at;
  __shared__ int failed_word, copied, given_up;  // steps copied; the first CTA's failed_word
  volatile int* failed = &failed_word;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const uint32_t full = smem_u32(bars), empty = full + 8 * kMaxSlots,
                 summed = full + 16 * kMaxSlots, drained = summed + 16,
                 idle = drained + 16;
  const uint32_t ring = smem_u32(smem);
  const uint32_t a_bytes = kTileM * kKStep * 2;
  const uint32_t b_bytes = static_cast<uint32_t>(p.half) * kKStep * 2;
  const uint32_t slot_bytes = a_bytes + b_bytes;
  const uint32_t rank = cluster_ctarank(), leader = 0;
  const int cluster = static_cast<int>(blockIdx.x) / 2, clusters = static_cast<int>(gridDim.x) / 2;
  const int tiles = p.m_tiles * p.n_tiles;
  if (warp == kWarpMma) {
    if (lane == 0) {
      for (int i = 0; i < p.slots; ++i) {
        mbar_init(full + 8 * i, 1);
        mbar_init(empty + 8 * i, 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(summed + 8 * i, 1);
        mbar_init(drained + 8 * i, 2 * kSumWarps);
      }
      mbar_init(idle, 1);
      *failed = 0;
      given_up = 0;
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc_pair(smem_u32(&tmem_at), 512);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync_all();  // the other's barriers and TMEM are there
  tc_fence_after();
  grid_dependency_wait();
  grid_dependents_go();
  const uint32_t tmem = tmem_at;
  // tile i in groups of eight tiles of tokens, whose rows stay in L2 while the
  // weight goes by
  const auto place = [&](int i, int* m, int* n) {
    constexpr int kGroup8 = 8;
    const int per = kGroup8 * p.n_tiles, group = i / per, rest = i - group * per;
    const int height = min(kGroup8, p.m_tiles - group * kGroup8);
    *n = rest / height;
    *m = group * kGroup8 + rest - *n * height;
  };

  // 384 threads have 168 registers each: the sums' 256 threads take 208, the others
  // keep 88 (256 * 208 + 128 * 88 = 384 * 168)
  if (warp < kSumWarps) {
    registers_up<208>();
    // lane + 32 (warp % 4) = token of the CTA, half of the output's columns: its sums
    // in registers, then 32 columns at a time through two tiles of 32 x 32 by
    // turns, into which the addend is copied two ahead (a load that is waited for
    // takes its turn behind the operands' copies: 4000 cycles)
    float* tiles_at = reinterpret_cast<float*>(smem + kRingBytes) + warp * (2 * 32 * kChunk);
    const int quarter = warp % 4, cols = p.out_cols / 2, side = warp / 4 * cols;
    const int row = lane >> 3, quad = lane & 7;  // of a store: four rows at a time
    const bool ahead = p.a.addend != nullptr && p.columns % 4 == 0;
    const int runs = (p.k_steps + p.run - 1) / p.run;
    Ring acc;
    bool ok = true;  // (for good: an accumulator's last phase but one looks like its next)
    for (int tile = cluster; tile < tiles; tile += clusters) {
      int m, n;
      place(tile, &m, &n);
      const int m0 = (2 * m + static_cast<int>(rank)) * kTileM;  // its own tokens from here on
      const int t0 = first_token(m0, p.a.tokens) + quarter * 32 + row;
      const int c0 = n * p.out_cols + side + quad * 4;
      // the rows of a store, four further on each, that are this CTA's own
      const long long at0 = static_cast<long long>(t0) * p.columns + c0, four = 4LL * p.columns;
      uint32_t own = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        own |= static_cast<uint32_t>(t0 + 4 * i >= m0 && t0 + 4 * i < p.a.tokens) << i;
      const auto fetch = [&](int c) {
        if (ahead && c * kChunk < cols) {
          const uint32_t to = smem_u32(tiles_at + (c & 1) * (32 * kChunk));
          const bool in = c0 + c * kChunk < p.columns;
          const float* from = p.a.addend + at0 + c * kChunk;
#pragma unroll
          for (int i = 0; i < 8; ++i, from += four)
            copy16_of(to + tile_at(4 * i + row, quad) * 4, from, in && (own >> i & 1u) ? 16 : 0);
        }
        copies_commit();
      };
      fetch(0);
      fetch(1);
      float sum[kGroups][16];
      for (int run = 0; run < runs; ++run) {
        const bool there = ring_wait<true>(summed + 8 * acc.slot, acc.phase, failed, p.wait_limit);
        ok = __all_sync(0xffffffffu, there) && ok;
        tc_fence_after();
        const uint32_t at =
            tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 256 * acc.slot + side;
        // gated: gates in the first groups, ups in the last. (Columns that a narrow
        // tile does not have are read as well, and not used.)
        const uint32_t up = p.a.gated ? static_cast<uint32_t>(p.half) : kGroups / 2 * 16;
        take_sums(sum, run == 0, kGroups, [&](int g) {
          return at + g / (kGroups / 2) * up + g % (kGroups / 2) * 16;
        });
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive_remote_relaxed(map_to_cta(drained + 8 * acc.slot, leader));
        acc.next(2);
      }
#pragma unroll
      for (int c = 0; c < kGroups / 2; ++c) {
        if (c * kChunk >= cols) break;
        if (c < kGroups / 4 && p.a.gated) {
          // (a lane's own choice, by the columns that its tile has: a token's result is
          // the same beside any other. 8192 tokens of 8192 x 512: 69 us, 81 without the
          // quick form)
          float least = 0.f;
#pragma unroll
          for (int i = 0; i < 32; ++i)  // (a side is a multiple of eight columns)
            if (c * kChunk + i / 8 * 8 < cols) least = fminf(least, sum[2 * c + i / 16][i % 16]);
          const bool near = least >= kNearGate;
          const auto gated = [&](auto form) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float& v = sum[2 * c + i / 16][i % 16];
              v = form(v, sum[(2 * c + i / 16 + kGroups / 2) % kGroups][i % 16]);
            }
          };
          if (near && p.a.f32_out)
            gated([](float g, float u) { return silu_times_near(g, u); });
          else if (near)
            gated([](float g, float u) { return silu_times_quick(g, u); });
          else
            gated([](float g, float u) { return silu_times(g, u); });
        }
        float* here = tiles_at + (c & 1) * (32 * kChunk);
        copies_wait<1>();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = sum[2 * c + i / 4][i % 4 * 4 + j];
          float4* at4 = reinterpret_cast<float4*>(here + tile_at(lane, i));
          float4 out = make_float4(v[0], v[1], v[2], v[3]);
          if (ahead) out = add4(out, *at4);
          const float nan = __uint_as_float(0x7FC00000u);
          *at4 = ok ? out : make_float4(nan, nan, nan, nan);
        }
        __syncwarp();
        const int column = c0 + c * kChunk;
        const bool in = c * kChunk + quad * 4 < cols && column < p.columns;
        const uint32_t rows = in ? own : 0u;
        const auto value = [&](int i) {
          return *reinterpret_cast<const float4*>(here + tile_at(4 * i + row, quad));
        };
        if (p.columns % 4 != 0) {
#pragma unroll 1
          for (int i = 0; i < 8; ++i)
            if (rows >> i & 1u)
              store_out(p, t0 + 4 * i, column, add4(value(i), load_addend(p, t0 + 4 * i, column)));
        } else if (p.a.f32_out) {
          float* to = static_cast<float*>(p.a.out) + at0 + c * kChunk;
#pragma unroll
          for (int i = 0; i < 8; ++i, to += four)
            if (rows >> i & 1u) *reinterpret_cast<float4*>(to) = value(i);
        } else {
          __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.a.out) + at0 + c * kChunk;
#pragma unroll
          for (int i = 0; i < 8; ++i, to += four)
            if (rows >> i & 1u) *reinterpret_cast<uint2*>(to) = bf16x4(value(i));
        }
        __syncwarp();
        fetch(c + 2);
      }
    }
  } else {
    registers_down<88>();
    if (warp == kWarpCopy) {
      if (elect_one()) {
        Ring r;
        bool ok = true;
        int issued = 0;
        for (int tile = cluster; tile < tiles && ok; tile += clusters) {
          int m, n;
          place(tile, &m, &n);
          const int m0 = first_token((2 * m + static_cast<int>(rank)) * kTileM, p.a.tokens);
          const int w0 = p.a.gated ? n * p.half + static_cast<int>(rank) * p.columns
                                   : (2 * n + static_cast<int>(rank)) * p.half;
          for (int k = 0; k < p.k_steps; ++k) {
            ok = ring_wait<true>(empty + 8 * r.slot, r.phase ^ 1u, failed, p.wait_limit);
            if (!ok) break;
            if (rank == 0) mbar_arrive_expect_tx(full + 8 * r.slot, 2 * slot_bytes);
            const uint32_t bar = map_to_cta(full + 8 * r.slot, leader);
            const uint32_t to = ring + r.slot * slot_bytes;
            tma_load_2d_pair(to, &p.x, k * kKStep, m0, bar);
            tma_load_2d_pair(to + a_bytes, &p.weight, k * kKStep, w0, bar);
            ++issued;
            r.next(p.slots);
          }
        }
        copied = issued;
      }
    } else if (warp == kWarpMma) {
      if (rank == 0 && elect_one()) {
        Ring r, acc;
        const uint32_t idesc = idesc_bf16(2 * kTileM, static_cast<uint32_t>(2 * p.half));
        bool ok = true;
        for (int tile = cluster; tile < tiles && ok; tile += clusters) {
          uint32_t d = 0;
          int left = 0;  // steps of this accumulator (a remainder would take 100 cycles of a step)
          for (int k = 0; k < p.k_steps; ++k) {
            const bool fresh = left == 0;
            if (fresh) {
              if (k > 0) {
                tc_commit_pair_mc(summed + 8 * acc.slot, 3u);
                acc.next(2);
              }
              ok = ring_wait<true>(drained + 8 * acc.slot, acc.phase ^ 1u, failed, p.wait_limit);
              if (!ok) break;
              d = tmem + 256 * acc.slot;
              left = p.run;
            }
            --left;
            ok = ring_wait<true>(full + 8 * r.slot, r.phase, failed, p.wait_limit);
            if (!ok) break;
            tc_fence_after();
            const uint32_t from = ring + r.slot * slot_bytes;
            const uint64_t ad = smem_desc_sw128_kmajor(from);
            const uint64_t bd = smem_desc_sw128_kmajor(from + a_bytes);
#pragma unroll
            for (int j = 0; j < kKStep / 16; ++j)  // 32 bytes further along k
              mma_bf16_ss_pair(d, ad + 2 * j, bd + 2 * j, idesc, !fresh || j > 0);
            tc_commit_pair_mc(empty + 8 * r.slot, 3u);
            r.next(p.slots);
          }
          if (ok) tc_commit_pair_mc(summed + 8 * acc.slot, 3u);
          acc.next(2);
        }
        tc_commit_pair_mc(idle, 3u);
        drain<true>(idle, 0);  // (behind the last sums it is as good as done)
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (rank == 0 && threadIdx.x == 0 && *failed) {
    given_up = 1;
    st_cluster_s32(map_to_cta(smem_u32(&given_up), 1), 1);
  }
  cluster_sync_all();  // nothing reaches across any more
  if (given_up) {
    // (else every copy has been multiplied.) The two may have stopped at different
    // steps: the first CTA, to which all copies report, expects what only the other
    // has copied, counts what that has not, and all that is under way lands.
    if (rank == 0 && threadIdx.x == 0) {
      const int other = ld_cluster_s32(map_to_cta(smem_u32(&copied), 1));
      const int end = max(copied, other);
      for (int i = max(0, end - p.slots); i < end; ++i) {
        const uint32_t bar = full + 8 * (i % p.slots);
        if (i >= copied) mbar_arrive_expect_tx(bar, slot_bytes);
        if (i >= other) mbar_complete_tx(bar, slot_bytes);
        drain<true>(bar, i / p.slots & 1);
      }
    }
    __syncwarp();
    cluster_sync_all();
  }
  if (warp == kWarpMma) {
    drain<true>(idle, 0);  // also of the second CTA: the last that the first sends it
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Where tiles are few: 128 tokens x 2 * half weight rows by a cluster whose CTAs
// split the columns of x. Their sums meet through the cluster's shared memory.
__global__ void __launch_bounds__(kDenseThreads, 1)
    w4a16_dense_split_kernel(const __grid_constant__ DenseArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t bars[2 * kMaxSlots + 5];
  __shared__ uint32_t tmem_at;
  __shared__ int failed_word;
  volatile int* failed = &failed_word;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const uint32_t full = smem_u32(bars), empty = full + 8 * kMaxSlots,
                 summed = full + 16 * kMaxSlots, drained = summed + 16,
                 idle = drained + 16;
  const uint32_t ring = smem_u32(smem);
  const uint32_t a_bytes = kTileM * kKStep * 2;
  const uint32_t b_bytes = static_cast<uint32_t>(p.half) * kKStep * 2;
  const uint32_t slot_bytes = a_bytes + 2 * b_bytes;
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / p.split;
  const int m = tile % p.m_tiles, n = tile / p.m_tiles;
  const int m0 = first_token(m * kTileM, p.a.tokens), skip = m * kTileM - m0;
  const int k0 = p.k_steps * rank / p.split, k1 = p.k_steps * (rank + 1) / p.split;
  const uint32_t acc_cols = p.half <= 32 ? 64 : p.half <= 64 ? 128 : 256, tmem_cols = 2 * acc_cols;
  const int w0 = p.a.gated ? n * p.half : 2 * n * p.half;
  const int w1 = w0 + (p.a.gated ? p.columns : p.half);
  // The first weights set out while the kernel before is at work (64 tokens 14.8 -> 14.3
  // us; for the pairs, whose first tile is a smaller part, it changes nothing).
  if (warp == kWarpCopy && elect_one())
    for (int k = k0; k < min(k1, k0 + p.slots); ++k) {
      prefetch_l2_2d(&p.weight, k * kKStep, w0);
      if (w1 < p.a.n) prefetch_l2_2d(&p.weight, k * kKStep, w1);
    }
  __syncwarp();
  if (warp == kWarpMma) {
    if (lane == 0) {
      for (int i = 0; i < p.slots; ++i) {
        mbar_init(full + 8 * i, 1);
        mbar_init(empty + 8 * i, 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(summed + 8 * i, 1);
        mbar_init(drained + 8 * i, kSumWarps);
      }
      mbar_init(idle, 1);
      *failed = 0;
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(smem_u32(&tmem_at), tmem_cols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();
  grid_dependents_go();
  const uint32_t tmem = tmem_at;
  bool ok = true;
  if (warp == kWarpCopy) {
    if (elect_one()) {
      Ring r;
      int k = k0;
      for (; k < k1; ++k) {
        ok = ring_wait<false>(empty + 8 * r.slot, r.phase ^ 1u, failed, p.wait_limit);
        if (!ok) break;
        const uint32_t to = ring + r.slot * slot_bytes, bar = full + 8 * r.slot;
        mbar_arrive_expect_tx(bar, slot_bytes);
        tma_load_2d(to + a_bytes, &p.weight, k * kKStep, w0, bar);
        tma_load_2d(to + a_bytes + b_bytes, &p.weight, k * kKStep, w1, bar);
        tma_load_2d(to, &p.x, k * kKStep, m0, bar);
        r.next(p.slots);
      }
      // copies in flight land before the CTA ends (they have, where all were multiplied)
      for (int i = max(0, k - k0 - p.slots); i < k - k0; ++i)
        drain<false>(full + 8 * (i % p.slots), i / p.slots & 1);
    }
  } else if (warp == kWarpMma) {
    if (elect_one()) {
      Ring r, acc;
      const uint32_t idesc = idesc_bf16(kTileM, static_cast<uint32_t>(2 * p.half));
      int left = 0;  // steps of this accumulator
      for (int k = k0; k < k1; ++k) {
        const bool fresh = left == 0;
        if (fresh) {
          if (k > k0) {
            tc_commit(summed + 8 * acc.slot);
            acc.next(2);
          }
          ok = ring_wait<false>(drained + 8 * acc.slot, acc.phase ^ 1u, failed, p.wait_limit);
          if (!ok) break;
          left = p.run;
        }
        --left;
        ok = ring_wait<false>(full + 8 * r.slot, r.phase, failed, p.wait_limit);
        if (!ok) break;
        tc_fence_after();
        const uint32_t from = ring + r.slot * slot_bytes;
        const uint64_t ad = smem_desc_sw128_kmajor(from);
        const uint64_t bd = smem_desc_sw128_kmajor(from + a_bytes);
#pragma unroll
        for (int j = 0; j < kKStep / 16; ++j)
          mma_bf16_ss(tmem + acc.slot * acc_cols, ad + 2 * j, bd + 2 * j, idesc, !fresh || j > 0);
        tc_commit(empty + 8 * r.slot);
        r.next(p.slots);
      }
      if (ok) tc_commit(summed + 8 * acc.slot);
      tc_commit(idle);
      drain<false>(idle, 0);
    }
  } else if (warp < kSumWarps) {
    // lane + 32 (warp % 4) = token of the tile, half of the weight rows
    const int quarter = warp % 4, side = warp / 4 * p.half, pitch = 2 * p.half + 4;
    const int runs = (k1 - k0 + p.run - 1) / p.run;
    float sum[kGroups][16];
    Ring acc;
    for (int run = 0; run < runs; ++run) {
      const bool there = ring_wait<false>(summed + 8 * acc.slot, acc.phase, failed, p.wait_limit);
      ok = __all_sync(0xffffffffu, there) && ok;
      tc_fence_after();
      const uint32_t at =
          tmem + (static_cast<uint32_t>(quarter * 32) << 16) + acc.slot * acc_cols + side;
      take_sums(sum, run == 0, p.half / 16, [&](int g) { return at + g * 16; });
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(drained + 8 * acc.slot);
      acc.next(2);
    }
    // (nothing reads the ring any more: all of its copies were multiplied)
    float* row = reinterpret_cast<float*>(smem) + (quarter * 32 + lane) * pitch + side;
    if (ok && m0 + quarter * 32 < p.a.tokens)  // (whole warps)
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
        if (g * 16 < p.half)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(row + g * 16 + i) =
                make_float4(sum[g][i], sum[g][i + 1], sum[g][i + 2], sum[g][i + 3]);
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
  const int pitch = 2 * p.half + 4, quads = p.out_cols / 4;
  if (*failed) {  // (only now that no copy is under way into this memory)
    for (int i = threadIdx.x; i < kTileM * pitch; i += kDenseThreads)
      reinterpret_cast<float*>(smem)[i] = __uint_as_float(0x7FC00000u);
    __syncthreads();
  }
  if (p.split > 1) cluster_sync_all();
  // every CTA of the cluster finishes a share of the tile, four columns a thread
  const int rows = min(kTileM, p.a.tokens - m * kTileM);
  const float* sums = reinterpret_cast<const float*>(smem);
  const int begin = rank * kDenseThreads + static_cast<int>(threadIdx.x);
  const int stride = p.split * kDenseThreads;
  const int r_step = stride / quads, q_step = stride - r_step * quads;
  int r = begin / quads + skip, q = begin % quads;
  for (; r < rows + skip; r += r_step, q += q_step) {
    if (q >= quads) {
      q -= quads;
      if (++r >= rows + skip) break;
    }
    const int c = 4 * q;
    const auto sum = [&](int column) {
      const float* at = sums + r * pitch + column;
      if (p.split == 1) return *reinterpret_cast<const float4*>(at);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s < p.split)
          v = add4(v, ld_cluster_f32x4(map_to_cta(smem_u32(at), static_cast<uint32_t>(s))));
      return v;
    };
    float4 v = sum(c);
    if (p.a.gated) {
      const float4 up = sum(p.half + c);
      v = make_float4(silu_times(v.x, up.x), silu_times(v.y, up.y), silu_times(v.z, up.z),
                      silu_times(v.w, up.w));
    }
    const int token = m0 + r, column = n * p.out_cols + c;
    store_out(p, token, column, add4(v, load_addend(p, token, column)));
  }
  if (p.split > 1) cluster_sync_all();  // the sums stay until all have read them
}

namespace {

int split_clusters_at_once(int ctas, int sms, int device, cudaError_t* error) {
  static ClustersAtOnce known[kMaxDenseSplit + 1];
  if (ctas == 1) return sms;
  return std::max(1, clusters_at_once(w4a16_dense_split_kernel, ctas, kDenseThreads, kSmemBytes,
                                      known[ctas], device, error));
}
int pairs_at_once(int device, cudaError_t* error) {
  static ClustersAtOnce known;
  return std::max(1, clusters_at_once(w4a16_dense_pair_kernel, 2, kDenseThreads, kSmemBytes, known,
                                      device, error));
}

// The faster kernel and its tile by an estimate in us: rounds of tiles times the
// steps of 64 columns of each, plus what a launch, the ring's first fill and the
// last tile's sums take. A step of a pair takes 270, 421, 540 and 590 cycles at 64,
// 128, 192 and 256 weight rows, its MMAs alone 128 to 512: what a CTA copies (16 KB
// of tokens and 64 bytes a weight row) goes into shared memory and out again at
// 128 to 150 bytes a cycle. (A second copying thread changes nothing, and L2 gives
// every SM 80 bytes a cycle.) Measured (gated, hidden 7168 x 4096, 64 / 576 / 2048
// tokens): split by 4 14.6 / 63 / 179, pairs of 192 44 / 38 / 92, pairs of 256 48 /
// 41 / 74 us. Pairs take widths in steps of 32 (2048 tokens: 224 rows 68 us, 256 73;
// 700 tokens, 7168 x 18432: 139 and 159), the split kernel, whose estimate is too low at
// 224 (400 tokens 31 us, pairs of 128 29), in steps of 64.
bool dense_shape(const ProductArgs& a, const DenseRoom& room, DenseArgs* best) {
  const int columns = a.gated ? a.n / 2 : a.n;
  const int steps = ceil_div(a.k, kKStep);
  double least = 0;
  bool pair = false;
  const auto consider = [&](const DenseArgs& c, bool is_pair, double cost) {
    if (least > 0 && cost >= least) return;
    least = cost;
    pair = is_pair;
    *best = c;
  };
  for (int tile_n = 64; tile_n <= 256; tile_n += 32) {
    DenseArgs c = {};
    c.columns = columns;
    c.half = tile_n / 2;
    c.out_cols = a.gated ? c.half : tile_n;
    c.n_tiles = ceil_div(columns, c.out_cols);
    c.k_steps = steps;
    // (BF16 results: equal runs, 17 steps as 9 and 8)
    const auto run = [&](int n) {
      return a.f32_out ? kRun : ceil_div(n, ceil_div(n, kRunRounded));
    };
    c.run = run(steps);
    const double gate = a.gated ? tile_n * 0.01 : 0;

    c.m_tiles = ceil_div(a.tokens, 2 * kTileM);
    c.split = 1;
    c.slots = std::min(kMaxSlots, kRingBytes / ((kTileM + c.half) * kKStep * 2));
    const double rounds = std::ceil(static_cast<double>(c.m_tiles) * c.n_tiles /
                                    room.pairs);
    consider(c, true, rounds * std::max(steps * (0.095 + tile_n * 0.00085), 2.0 + tile_n * 0.008) +
                          5 + tile_n * 0.01 + gate);

    if (tile_n % 64 != 0) continue;
    c.m_tiles = ceil_div(a.tokens, kTileM);
    c.slots = std::min(kMaxSlots, kRingBytes / ((kTileM + tile_n) * kKStep * 2));
    const double rows = std::min(a.tokens, kTileM);
    for (c.split = 1; c.split <= kMaxDenseSplit && c.split <= steps; c.split *= 2) {
      if (static_cast<long long>(c.m_tiles) * c.n_tiles * c.split > 0x7fffffffLL) break;
      const double waves = std::ceil(static_cast<double>(c.m_tiles) * c.n_tiles /
                                     room.clusters[c.split]);
      c.run = run(ceil_div(steps, c.split));
      const double sums = rows / kTileM * (1 + tile_n * 0.012 + gate) / (c.split > 1 ? 1.5 : 1);
      consider(c, false, waves * (ceil_div(steps, c.split) * (0.07 + tile_n * 0.00125) + 4.5 +
                                  (c.split > 1 ? 1.5 : 0) + sums));
    }
  }
  return pair;
}

}  // namespace

cudaError_t dense_room(int sms, DenseRoom* room) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device >= kMaxDevices) return cudaErrorInvalidDevice;
  room->pairs = pairs_at_once(device, &e);
  for (int split = 1; split <= kMaxDenseSplit; split *= 2)
    room->clusters[split] = split_clusters_at_once(split, sms, device, &e);
  return e;
}

DenseShape dense_choice(const ProductArgs& args, const DenseRoom& room) {
  if (args.tokens <= kDenseFewTokens) return {};
  DenseArgs p;
  const bool pair = dense_shape(args, room, &p);
  return {pair ? 2 : 1, 2 * p.half, p.split, p.run * kKStep};
}

cudaError_t launch_dense(const ProductArgs& args, int sms, cudaStream_t stream) {
  if (args.tokens <= kDenseFewTokens) return launch_dense_few(args, sms, stream);
  DenseRoom room;
  cudaError_t e = dense_room(sms, &room);
  if (e != cudaSuccess) return e;
  DenseArgs p;
  const bool pair = dense_shape(args, room, &p);
  p.a = args;
  p.wait_limit = wait_timeout_cycles();
  if (!encode_rows_tmap(&p.x, args.x, args.tokens, args.k, args.x_stride, kTileM) ||
      !encode_rows_tmap(&p.weight, args.weight, args.n, args.k, args.k, p.half))
    return cudaErrorInvalidValue;
  const long long tiles = static_cast<long long>(p.m_tiles) * p.n_tiles;
  static Devices known[2];
  e = allow_smem(pair ? w4a16_dense_pair_kernel : w4a16_dense_split_kernel, kSmemBytes,
                 known[pair ? 1 : 0]);
  if (e != cudaSuccess) return e;
  if (pair) {
    const int clusters = static_cast<int>(std::min<long long>(tiles, room.pairs));
    return launch_dependent(w4a16_dense_pair_kernel, 2 * clusters, kDenseThreads, kSmemBytes, 2,
                            stream, p);
  }
  const int smem = 1024 + std::max(p.slots * (kTileM + 2 * p.half) * kKStep * 2,
                                   kTileM * (2 * p.half + 4) * 4);
  return launch_dependent(w4a16_dense_split_kernel, static_cast<int>(tiles) * p.split,
                          kDenseThreads, static_cast<size_t>(smem), p.split, stream, p);
}

}  // namespace w4a16
