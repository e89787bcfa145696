// router.cu -- the router's product: logits = x . weight^T, BF16 operands,
// FP32 sums.
//
// Two kernels, by the number of tokens:
//
//   * few, as long as all of its CTAs run at once (64 tokens of 384 experts, 400
//     of 60): a cluster of up to eight CTAs shares sixteen experts and 32 tokens,
//     each CTA a share of the columns, so that all SMs read a part of the weight
//     (5.5 MB for 384 experts of hidden 7168) at once; m16n8k16 MMAs straight
//     from global memory (no operand is used twice by a CTA), partial sums
//     joined through the cluster's shared memory;
//   * more: a dense product on tcgen05, 128 tokens (256 of a CTA pair) x up to
//     256 experts a tile, both operands by TMA, accumulators in TMEM. Where the
//     tiles are fewer than the SMs, a cluster of up to eight CTAs splits the
//     columns of one.
//
// The order of the additions follows from the sizes and from how many clusters
// the device runs at once.
//
// 384 experts of hidden 7168, in a graph: 1 token 3.2 us, 48 tokens 6.5 us, both
// latency (launch, one round of loads, two for 48 tokens, the cluster's exchange;
// the weight alone is 0.8 us of the copy rate). 8192 tokens: 40 us, 1.1 PFLOP/s, 0.59 of a
// library product's rate, on 128 of 152 SMs: 7 us are launch, first loads and
// the logits' way out, the rest is bound by the operands' way into an SM
// (28 KB of 64 columns at 50 bytes a cycle, against 384 cycles of MMAs).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace w4a16 {

namespace {

// ----------------------------------------------------------- few tokens ---

constexpr int kFewBlock = 32;  // tokens of a CTA at most (64: 9.9 us for 48 tokens, 32: 6.5)
constexpr int kFewWarps = 8;
constexpr int kFewExperts = 16;  // of a cluster (MMA M)

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace

// kNt tiles of eight tokens, clusters of kCl CTAs. Columns go in blocks of 32: thread t of a quad
// takes columns 8t .. 8t + 7 of a block, of both operands alike, so one 16-byte
// load a row feeds two MMAs whatever order the MMA gives its k.
template <int kNt, int kCl>
__global__ void __launch_bounds__(kFewWarps * 32)
    w4a16_router_few_kernel(const uint16_t* __restrict__ x, long long x_stride,
                            const uint16_t* __restrict__ weight, int tokens, int hidden,
                            int num_experts, float* __restrict__ logits) {
  __shared__ float part[kFewWarps][kFewExperts * 8 * kNt];
  __shared__ float sums[kFewExperts * 8 * kNt];  // [token][expert]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(cluster_ctarank());
  const int tile = static_cast<int>(blockIdx.x) / kCl;
  const int e_tiles = (num_experts + kFewExperts - 1) / kFewExperts;
  const int e0 = tile % e_tiles * kFewExperts;
  const int t0 = tile / e_tiles * (8 * kNt);
  x += t0 * x_stride;
  logits += static_cast<long long>(t0) * num_experts;
  tokens = min(tokens - t0, 8 * kNt);
  grid_dependency_wait();
  grid_dependents_go();
  const int blocks = (hidden + 31) / 32;
  const int first = blocks * rank / kCl, last = blocks * (rank + 1) / kCl;
  const uint16_t* a0 = weight + static_cast<long long>(min(e0 + g, num_experts - 1)) * hidden;
  const uint16_t* a1 = weight + static_cast<long long>(min(e0 + g + 8, num_experts - 1)) * hidden;
  const uint16_t* b[kNt];
#pragma unroll
  for (int n = 0; n < kNt; ++n) b[n] = x + min(8 * n + g, tokens - 1) * x_stride;
  float acc[kNt][4] = {};
  constexpr int kUnroll = kNt <= 2 ? 4 : 2;  // blocks in flight
  for (int blk = first + warp; blk < last; blk += kFewWarps * kUnroll) {
    uint4 va[kUnroll][2], vb[kUnroll][kNt];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int k = (blk + u * kFewWarps) * 32 + t * 8;
      const bool in = blk + u * kFewWarps < last && k < hidden;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      va[u][0] = in ? __ldg(reinterpret_cast<const uint4*>(a0 + k)) : zero;
      va[u][1] = in ? __ldg(reinterpret_cast<const uint4*>(a1 + k)) : zero;
#pragma unroll
      for (int n = 0; n < kNt; ++n)
        vb[u][n] = in ? __ldg(reinterpret_cast<const uint4*>(b[n] + k)) : zero;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int n = 0; n < kNt; ++n) {
        mma_bf16(acc[n], va[u][0].x, va[u][1].x, va[u][0].y, va[u][1].y, vb[u][n].x, vb[u][n].y);
        mma_bf16(acc[n], va[u][0].z, va[u][1].z, va[u][0].w, va[u][1].w, vb[u][n].z, vb[u][n].w);
      }
  }
#pragma unroll
  for (int n = 0; n < kNt; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      part[warp][(8 * n + 2 * t + (i & 1)) * kFewExperts + g + (i >> 1) * 8] = acc[n][i];
  __syncthreads();
  for (int i = threadIdx.x; i < kFewExperts * 8 * kNt; i += kFewWarps * 32) {
    float v = part[0][i];
#pragma unroll
    for (int w = 1; w < kFewWarps; ++w) v += part[w][i];
    sums[i] = v;
  }
  cluster_sync_all();
  // every CTA of the cluster writes its share of the outputs
  for (int i = rank * kFewWarps * 32 + static_cast<int>(threadIdx.x); i < kFewExperts * tokens;
       i += kCl * kFewWarps * 32) {
    const int tok = i / kFewExperts, e = e0 + i % kFewExperts;
    const uint32_t at = smem_u32(sums + i);
    float v = 0.f;
#pragma unroll
    for (int c = 0; c < kCl; ++c)
      v += ld_cluster_f32(map_to_cta(at, static_cast<uint32_t>(c)));
    if (e < num_experts) logits[static_cast<long long>(tok) * num_experts + e] = v;
  }
  cluster_sync_all();  // the sums stay until all have read them
}

namespace {

// ---------------------------------------------------------- many tokens ---

constexpr int kTileM = 128;        // tokens of a tile (MMA M)
constexpr int kMaxTileN = 256;     // experts of a tile (MMA N)
constexpr int kMaxSplit = 8;
constexpr int kMaxRing = 8;
constexpr int kRingBytes = 224 << 10;
// Eight epilogue warps, then two that copy and two that issue MMAs, by turns:
// one thread gets round its loop (wait, copy or multiply, report) only every
// 600 to 1100 cycles, against 384 of a k step at N = 192 (8192 tokens: 67 us
// with one of each).
constexpr int kDensePairs = 2;
constexpr int kSumWarps = 8;       // two a TMEM quarter, half of the columns each
constexpr int kDenseThreads = 32 * (kSumWarps + 2 * kDensePairs);
constexpr int kWarpCopy0 = kSumWarps, kWarpMma0 = kSumWarps + kDensePairs;
// The tensor core cuts its sums off instead of rounding them, which over the
// 224 additions that 7168 columns are to each of two accumulators came to
// 3.8e-6 of the logits. So after 512 columns (32 additions) an MMA thread
// hands its accumulator to the epilogue warps, which add it to FP32 sums in
// registers, and begins at zero: 4.8e-7, for 2 us of 50.
constexpr int kChunk = 8;  // times kKStep columns
constexpr long long kGiveUpCycles = 4000000000LL;  // about two seconds

struct DenseArgs {
  CUtensorMap x, weight;
  float* logits;
  int tokens, num_experts;
  int k_steps, sub;  // steps of sub * kKStep columns
  int tile_n, b_rows, n_tiles, split, slots, tmem_cols;
};

// Ring slots, a multiple of the threads that take turns: each slot then belongs
// to one copy and one MMA thread. (In a ring of five a thread could come to a
// slot two phases ahead of it, which a wait on the phase's parity cannot tell
// from done.) 4 of 128 columns in a pair at N = 192, 6 of 64 at N = 256, 4 to 8
// of 64 of one CTA.
int dense_slots(int b_rows, int sub) {
  const int fit = std::min(kMaxRing, kRingBytes / ((kTileM + b_rows) * sub * kKStep * 2));
  return fit / kDensePairs * kDensePairs;
}
// The ring's memory, which the swizzle wants at 1024 bytes, is later the tile's
// sums [token][expert], four floats between rows so that they start on
// different banks, and behind them what the other CTAs of a split send.
__host__ __device__ inline int sum_pitch(int tile_n) { return tile_n + 4; }
__host__ __device__ inline int tile_sums_bytes(int tile_n) {
  return kTileM * sum_pitch(tile_n) * 4;
}
size_t dense_smem(const DenseArgs& a) {
  const size_t ring = static_cast<size_t>(a.slots) * (kTileM + a.b_rows) * a.sub * kKStep * 2;
  const size_t sums = static_cast<size_t>(tile_sums_bytes(a.tile_n)) * (a.split > 1 ? 2 : 1);
  return 2048 + std::max(ring, sums);
}

// kRemote: threads of the other CTA of a pair arrive as well.
template <bool kRemote = false>
__device__ __forceinline__ bool dense_wait(uint32_t bar, uint32_t parity, volatile int* failed) {
  const long long t0 = clock64();
  while (!(kRemote ? mbar_try_wait_cluster_now(bar, parity) : mbar_try_wait(bar, parity))) {
    if (*failed) return false;
    if (clock64() - t0 > kGiveUpCycles) {
      *failed = 1;
      return false;
    }
  }
  return true;
}

}  // namespace

// kPair: two CTAs multiply a tile of 256 tokens together. Each copies its own
// 128 tokens and half of the experts, 28 KB of 64 columns at N = 192 instead of
// 40, all copies report to the first CTA, whose MMA threads issue for both, and
// every CTA keeps the sums of its tokens. Otherwise a tile has 128 tokens and
// one CTA. a.split CTAs or pairs of a cluster share a tile by its columns.
// A wait that gives up (none does unless the hardware fails) ends the CTA's
// work in order and leaves NaN in its logits.
// kSub * kKStep columns are a step (of a constant count: a loop over a variable
// one cost the MMA threads 0.6 us of 777 tokens' 7.7).
template <bool kPair, int kSub>
__global__ void __launch_bounds__(kDenseThreads, 1)
    w4a16_router_dense_kernel(const __grid_constant__ DenseArgs a) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t bars[2 * kMaxRing + 2 * kDensePairs + 1];
  __shared__ uint32_t tmem_at;
  __shared__ int failed_word;
  volatile int* failed = &failed_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t full = smem_u32(bars), empty = full + 8 * kMaxRing, done = full + 16 * kMaxRing,
                 drained = done + 8 * kDensePairs, received = drained + 8 * kDensePairs;
  const uint32_t ring = smem_u32(smem);
  const uint32_t a_bytes = kTileM * kKStep * 2, b_bytes = static_cast<uint32_t>(a.b_rows) * kKStep * 2;
  const uint32_t sub_bytes = a_bytes + b_bytes, slot_bytes = sub_bytes * kSub;
  const int ctas = (kPair ? 2 : 1) * a.split;  // of a tile
  const int id = static_cast<int>(blockIdx.x) % ctas;  // in the cluster
  const int half = kPair ? id & 1 : 0, rank = kPair ? id >> 1 : id;  // of the tokens, columns
  const uint32_t leader = static_cast<uint32_t>(kPair ? id & ~1 : id);
  constexpr int kRun = kChunk / kSub;
  const int tile = static_cast<int>(blockIdx.x) / ctas;
  const int m0 = (kPair ? tile / a.n_tiles * 2 + half : tile / a.n_tiles) * kTileM;
  const int n0 = tile % a.n_tiles * a.tile_n;
  const int k0 = a.k_steps * rank / a.split, k1 = a.k_steps * (rank + 1) / a.split;
  if (warp == kWarpMma0) {
    if (lane == 0) {
      for (int i = 0; i < a.slots; ++i) {
        mbar_init(full + 8 * i, 1);
        mbar_init(empty + 8 * i, 1);
      }
      for (int i = 0; i < kDensePairs; ++i) {
        mbar_init(done + 8 * i, 1);
        mbar_init(drained + 8 * i, kPair ? 2 * kSumWarps : kSumWarps);
      }
      mbar_init(received, 1);
      *failed = 0;
      fence_mbar_init();
    }
    __syncwarp();
    if constexpr (kPair) {
      tmem_alloc_pair(smem_u32(&tmem_at), static_cast<uint32_t>(a.tmem_cols));
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&tmem_at), static_cast<uint32_t>(a.tmem_cols));
      tmem_relinquish();
    }
    tc_fence_before();
  }
  __syncthreads();
  if constexpr (kPair) cluster_sync_all();  // the other's barriers and TMEM are there
  tc_fence_after();
  grid_dependency_wait();
  grid_dependents_go();
  const uint32_t tmem = tmem_at;

  if (warp >= kWarpCopy0 && warp < kWarpMma0) {
    if (lane == 0) {
      bool ok = true;
      const int first = warp - kWarpCopy0;
      int issued = first;  // k step of this CTA
      for (; k0 + issued < k1; issued += kDensePairs) {
        const int slot = issued % a.slots, k = k0 + issued;
        ok = dense_wait(empty + 8 * slot, (issued / a.slots & 1) ^ 1, failed);
        if (!ok) break;
        if (half == 0)
          mbar_arrive_expect_tx(full + 8 * slot, kPair ? 2 * slot_bytes : slot_bytes);
#pragma unroll
        for (int j = 0; j < kSub; ++j) {
          const uint32_t to = ring + slot * slot_bytes + j * sub_bytes;
          const int column = (k * kSub + j) * kKStep;
          if constexpr (kPair) {
            const uint32_t bar = map_to_cta(full + 8 * slot, leader);
            tma_load_2d_pair(to, &a.x, column, m0, bar);
            tma_load_2d_pair(to + a_bytes, &a.weight, column, n0 + half * a.b_rows, bar);
          } else {
            tma_load_2d(to, &a.x, column, m0, full + 8 * slot);
            tma_load_2d(to + a_bytes, &a.weight, column, n0, full + 8 * slot);
          }
        }
      }
      if (!ok && half == 0)  // copies in flight land before the CTAs end
        for (int i = first; i < issued; i += kDensePairs) {
          if (i < issued - a.slots) continue;
          const long long t0 = clock64();
          while (!mbar_try_wait(full + 8 * (i % a.slots), i / a.slots & 1) &&
                 clock64() - t0 < kGiveUpCycles) {
          }
        }
    }
  } else if (warp >= kWarpMma0) {
    // each into an accumulator of its own
    if (lane == 0 && half == 0) {
      const auto report = [&](uint32_t bar) {
        if constexpr (kPair)
          tc_commit_pair_mc(bar, static_cast<uint16_t>(3u << leader));
        else
          tc_commit(bar);
      };
      const int first = warp - kWarpMma0;
      const uint32_t d = tmem + static_cast<uint32_t>(first * a.tmem_cols / kDensePairs);
      const uint32_t idesc = idesc_bf16(kPair ? 2 * kTileM : kTileM, static_cast<uint32_t>(a.tile_n));
      bool ok = true;
      int n = 0;  // steps of this thread
      for (int i = first; k0 + i < k1; i += kDensePairs, ++n) {
        const int slot = i % a.slots;
        if (n > 0 && n % kRun == 0) {
          report(done + 8 * first);
          ok = dense_wait<kPair>(drained + 8 * first, (n / kRun - 1) & 1, failed);
          if (!ok) break;
          tc_fence_after();
        }
        ok = dense_wait(full + 8 * slot, i / a.slots & 1, failed);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          const uint32_t from = ring + slot * slot_bytes + u * sub_bytes;
          const uint64_t ad = smem_desc_sw128_kmajor(from);
          const uint64_t bd = smem_desc_sw128_kmajor(from + a_bytes);
#pragma unroll
          for (int j = 0; j < kKStep / 16; ++j) {  // 32 bytes further along k
            const uint32_t add = n % kRun != 0 || u > 0 || j > 0;
            if constexpr (kPair)
              mma_bf16_ss_pair(d, ad + 2 * j, bd + 2 * j, idesc, add);
            else
              mma_bf16_ss(d, ad + 2 * j, bd + 2 * j, idesc, add);
          }
        }
        report(empty + 8 * slot);
      }
      if (n > 0 && ok) report(done + 8 * first);
    }
  } else {
    // lane + 32 (warp % 4) = token of the tile, half of the experts; in the end
    // the sums take the ring's place
    const int left = (a.tile_n / 2 + 15) / 16 * 16;
    const int c0 = warp < 4 ? 0 : left, cols = warp < 4 ? left : a.tile_n - left;
    const uint32_t at = tmem + (static_cast<uint32_t>(warp % 4 * 32) << 16) + c0;
    float sum[kMaxTileN / 2] = {};
    bool ok = true;
    for (int c = 0; ok; ++c) {
      bool any = false;
      for (int j = 0; j < kDensePairs && ok; ++j) {
        // chunk c of MMA thread j, which has the steps j, j + kDensePairs, ...
        if (j + c * kRun * kDensePairs >= k1 - k0) continue;
        any = true;
        ok = __all_sync(0xffffffffu, dense_wait(done + 8 * j, c & 1, failed));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int p = 0; p < kMaxTileN / 32; ++p)
          if (16 * p < cols) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(at + j * (a.tmem_cols / kDensePairs) + 16 * p, v);
            tmem_ld_wait_for(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[16 * p + i] += __uint_as_float(v[i]);
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair)
            mbar_arrive_remote_relaxed(map_to_cta(drained + 8 * j, leader));
          else
            mbar_arrive(drained + 8 * j);
        }
      }
      if (!any) break;
    }
    ok = __all_sync(0xffffffffu, ok && !*failed);
    // (nothing reads the ring any more: all of its copies were multiplied)
    float* row = reinterpret_cast<float*>(smem) + (warp % 4 * 32 + lane) * sum_pitch(a.tile_n) + c0;
#pragma unroll
    for (int p = 0; p < kMaxTileN / 8; ++p)
      if (4 * p < cols)
        *reinterpret_cast<float4*>(row + 4 * p) =
            ok ? make_float4(sum[4 * p], sum[4 * p + 1], sum[4 * p + 2], sum[4 * p + 3])
               : make_float4(__uint_as_float(0x7FC00000u), __uint_as_float(0x7FC00000u),
                             __uint_as_float(0x7FC00000u), __uint_as_float(0x7FC00000u));
    fence_proxy_async_smem();  // a bulk copy sends them on
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if constexpr (kPair) cluster_sync_all();  // nothing reaches across any more
  if (warp == kWarpMma0) {
    tc_fence_after();
    if constexpr (kPair)
      tmem_dealloc_pair(tmem, static_cast<uint32_t>(a.tmem_cols));
    else
      tmem_dealloc(tmem, static_cast<uint32_t>(a.tmem_cols));
  }
  // a split: every CTA finishes a share of the tokens, whose sums the others
  // send it, one bulk copy each
  const int rows = kTileM / a.split, pitch = sum_pitch(a.tile_n);
  const uint32_t share = static_cast<uint32_t>(rows * pitch * 4);
  const uint32_t inbox = ring + static_cast<uint32_t>(tile_sums_bytes(a.tile_n));
  bool whole = true;
  if (a.split > 1) {
    if (threadIdx.x == 0) mbar_arrive_expect_tx(received, share * (a.split - 1));
    cluster_sync_all();  // everybody's ring is done with, and expects
    if (static_cast<int>(threadIdx.x) < a.split && static_cast<int>(threadIdx.x) != rank) {
      const uint32_t to = threadIdx.x, cta = kPair ? 2 * to + half : to;
      asm volatile(
          "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes "
          "[%0], [%1], %2, [%3];" ::"r"(map_to_cta(inbox + rank * share, cta)),
          "r"(ring + to * share), "r"(share), "r"(map_to_cta(received, cta))
          : "memory");
    }
    whole = dense_wait(received, 0, failed);
  }
  const float* sums = reinterpret_cast<const float*>(smem);
  const float* others = reinterpret_cast<const float*>(smem + (inbox - ring));
  const int n_end = min(a.tile_n, a.num_experts - n0);
  for (int r = warp; r < rows; r += kDenseThreads / 32) {
    const int m = rank * rows + r;
    if (m0 + m >= a.tokens) break;
    float* out = a.logits + static_cast<long long>(m0 + m) * a.num_experts + n0;
    if (a.split == 1) {
#pragma unroll 8
      for (int n = lane; n < n_end; n += 32) out[n] = sums[m * pitch + n];
      continue;
    }
    for (int n = lane; n < n_end; n += 32) {
      float v = 0.f;
      for (int c = 0; c < a.split; ++c)  // in the CTAs' order
        v += c == rank ? sums[m * pitch + n] : others[(c * rows + r) * pitch + n];
      out[n] = whole ? v : __uint_as_float(0x7FC00000u);
    }
  }
  if (a.split > 1) cluster_sync_all();  // the sums stay until all are sent
}

namespace {

// How many clusters of a kernel run at once, by device (0: not asked yet).
constexpr int kMaxDevices = 64;
using ClustersAtOnce = std::atomic<int>[kMaxDevices];

// How many clusters of `ctas` run at once on the current device (they stay
// inside a GPC, so eights of one CTA an SM leave some SMs out). 0 and an error
// if that cannot be said: a guess would let the same sizes take another order
// of additions in one call than in the next.
template <typename Kernel>
int clusters_at_once(Kernel kernel, int ctas, int threads, size_t smem, ClustersAtOnce& known,
                     int device, cudaError_t* error) {
  if (const int n = known[device]) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(ctas);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  cudaError_t e = cudaSuccess;
  if (smem > 0)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
  if (e != cudaSuccess) {
    *error = e;
    return 0;
  }
  known[device] = n;
  return n;
}

int dense_clusters_at_once(int ctas, int sms, int device, cudaError_t* error) {
  static ClustersAtOnce known[kMaxSplit + 1];
  if (ctas == 1) return sms;
  return std::max(1, clusters_at_once(w4a16_router_dense_kernel<false, 1>, ctas, kDenseThreads,
                                      kRingBytes + 2048, known[ctas], device, error));
}

// The fastest shape by an estimate in cycles: waves of clusters, each a CTA's
// steps at the rate at which an SM takes operands from L2 (50 bytes a cycle
// were measured) or at which the threads get round their loops, plus the
// tile's sums on their way out. Against every shape timed (65 to 8192 tokens of
// six weights) the choice is within 2 per cent of the fastest in the mean, 14
// at most; hidden 7168 x 384 experts, us: 777 tokens 17 (a pair of 128 experts,
// split by 4: 16; one CTA, split by 4: 18), 4096 tokens 28 (pairs unsplit 35,
// one CTA 33), 8192 tokens 40 (one CTA 54).
double dense_shape(int tokens, int num_experts, int hidden, int sms, int device, DenseArgs* a,
                   bool* best_pair, cudaError_t* error) {
  double best = 0;
  for (int pair = 0; pair < 2; ++pair)
    for (int width = 64; width <= kMaxTileN; width += 64) {
      DenseArgs c = {};
      const int step = pair ? 32 : 16;  // of an MMA's N
      c.n_tiles = ceil_div(num_experts, width);
      c.tile_n = ceil_div(ceil_div(num_experts, c.n_tiles), step) * step;
      c.b_rows = pair ? c.tile_n / 2 : c.tile_n;
      // 128 columns a step where four fit
      c.sub = pair && dense_slots(c.b_rows, 2) >= 4 ? 2 : 1;
      c.k_steps = ceil_div(hidden, c.sub * kKStep);
      c.slots = dense_slots(c.b_rows, c.sub);
      c.tmem_cols = 32;
      while (c.tmem_cols < c.tile_n * kDensePairs) c.tmem_cols *= 2;
      const double step_cycles =
          std::max(c.sub * (kTileM + c.b_rows) * kKStep * 2 / 50.0, c.sub == 1 ? 510.0 : 880.0);
      const double tiles =
          static_cast<double>(ceil_div(tokens, pair ? 2 * kTileM : kTileM)) * c.n_tiles;
      for (c.split = 1; c.split * (pair ? 2 : 1) <= kMaxSplit && c.split <= c.k_steps; c.split *= 2) {
        if (c.split > 1 && 2 * tile_sums_bytes(c.tile_n) > kRingBytes) break;
        const int ctas = c.split * (pair ? 2 : 1);
        const double waves = std::ceil(tiles / dense_clusters_at_once(ctas, sms, device, error));
        const double cost = waves * (ceil_div(c.k_steps, c.split) * step_cycles + 3000 +
                                     c.tile_n * 28 + (c.split == 1 ? 0 : pair ? 4500 : 3500));
        if (best == 0 || cost < best) {
          best = cost;
          *best_pair = pair != 0;
          *a = c;
        }
      }
    }
  return best;
}

// One wave of the few-token kernel is faster than the dense one and two are
// not, so its clusters are the largest that all run at once, if the columns
// that a CTA then has (2200 ns and 4.7 a column) take less than the dense kernel
// needs and, in clusters that have been made smaller, are not more than some
// 1100 (7168 x 16, 2000 tokens on fours: 14.5 us against 11.0). Hidden 7168 x 384 experts, 64 tokens (48 clusters of eight, 51
// run at once) 6.4 us against 9.0, 65 tokens 10.6 against 9.0; 2088 x 60, 192
// tokens 3.8 against 7.6, 777 tokens (fours) 6.2 against 7.8; 7168 x 1024, 16
// tokens (64 of 74) 5.6 against 10.8; 256 x 64, 2000 tokens 3.4 against 6.1.
template <int kNt, int kCl>
bool few_fits(long long clusters, int hidden, double dense_cycles, int device,
              cudaError_t* error) {
  static ClustersAtOnce known;
  return clusters <= clusters_at_once(w4a16_router_few_kernel<kNt, kCl>, kCl, kFewWarps * 32, 0,
                                      known, device, error) &&
         (kCl == 8 || hidden <= 1100 * kCl) &&
         4200 + 9.0 * hidden / kCl < dense_cycles + 2900;
}

}  // namespace

cudaError_t launch_router_logits(const uint16_t* x, long long x_stride, const uint16_t* weight,
                                 int tokens, int hidden, int num_experts, float* logits, int sms,
                                 cudaStream_t stream) {
  DenseArgs a;
  bool pair = false;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device >= kMaxDevices) return cudaErrorInvalidDevice;
  const double dense = dense_shape(tokens, num_experts, hidden, sms, device, &a, &pair, &e);
  const long long clusters =
      static_cast<long long>(ceil_div(num_experts, kFewExperts)) * ceil_div(tokens, kFewBlock);
  const auto few = [&](auto kernel, int ctas) {
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, static_cast<int>(clusters) * ctas, kFewWarps * 32, 0, ctas,
                            stream, x, x_stride, weight, tokens, hidden, num_experts, logits);
  };
  constexpr int kNt = kFewBlock / 8;
  if (tokens <= 8 && few_fits<1, 8>(clusters, hidden, dense, device, &e))
    return few(w4a16_router_few_kernel<1, 8>, 8);
  if (tokens <= 16 && few_fits<2, 8>(clusters, hidden, dense, device, &e))
    return few(w4a16_router_few_kernel<2, 8>, 8);
  if (few_fits<kNt, 8>(clusters, hidden, dense, device, &e))
    return few(w4a16_router_few_kernel<kNt, 8>, 8);
  if (few_fits<kNt, 4>(clusters, hidden, dense, device, &e))
    return few(w4a16_router_few_kernel<kNt, 4>, 4);
  if (few_fits<kNt, 2>(clusters, hidden, dense, device, &e))
    return few(w4a16_router_few_kernel<kNt, 2>, 2);
  if (few_fits<kNt, 1>(clusters, hidden, dense, device, &e))
    return few(w4a16_router_few_kernel<kNt, 1>, 1);
  if (e != cudaSuccess) return e;
  a.logits = logits;
  a.tokens = tokens;
  a.num_experts = num_experts;
  if (!encode_rows_tmap(&a.x, x, tokens, hidden, x_stride, kTileM) ||
      !encode_rows_tmap(&a.weight, weight, num_experts, hidden, hidden, a.b_rows))
    return cudaErrorInvalidValue;
  const int ctas = (pair ? 2 : 1) * a.split;
  const long long grid =
      static_cast<long long>(ceil_div(tokens, pair ? 2 * kTileM : kTileM)) * a.n_tiles * ctas;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  const auto kernel = !pair ? w4a16_router_dense_kernel<false, 1>
                      : a.sub == 1 ? w4a16_router_dense_kernel<true, 1>
                                   : w4a16_router_dense_kernel<true, 2>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kRingBytes + 2048);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, static_cast<int>(grid), kDenseThreads, dense_smem(a), ctas,
                          stream, a);
}

}  // namespace w4a16
