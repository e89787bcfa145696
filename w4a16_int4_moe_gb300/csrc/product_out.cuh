// product_out.cuh -- what the kernels of products for few tokens share: codes to
// numbers, scaled sums, and the sums' way out.
#pragma once

#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"
#include "silu.cuh"

namespace w4a16 {

namespace {

constexpr int kMaxSmem = 232448;
constexpr int kSumPad = 4;  // of a token's row of sums, so that rows start at other banks

__device__ __forceinline__ uint4 load_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// A BF16 number in shared memory.
__device__ __forceinline__ float load_scale(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// Two codes, in bits 3 to 6 of each half word, as BF16 numbers q - 8: in those bits
// of the number 16 a code is 16 + q, and both steps are exact. (sixteens is an
// argument so that the compiler keeps one three-input operation: with two
// constants it makes two of them, and 16384 x 7168 takes 18.8 instead of 16.1 us
// for one token.)
__device__ __forceinline__ uint32_t code_pair(uint32_t shifted, uint32_t sixteens) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(shifted), "r"(0x00780078u), "r"(sixteens));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0x41C041C0u));
  return r;
}

// d0 += s * c0, d1 += s * c1 in one operation
__device__ __forceinline__ void fma_pair(float& d0, float& d1, float s, float c0, float c1) {
  asm("{\n\t.reg .b64 c, s, d;\n\t"
      "mov.b64 c, {%3, %4};\n\tmov.b64 s, {%2, %2};\n\tmov.b64 d, {%0, %1};\n\t"
      "fma.rn.f32x2 d, s, c, d;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(s), "f"(c0), "f"(c1));
}

// The outputs begin, begin + stride, ... of a block of kRows weight rows, of the
// sums in part, [tokens][kRows + kSumPad], added over the cluster's `split` CTAs.
template <bool kGated, int kRows>
__device__ __forceinline__ void write_products(const ProductArgs& a, const float* part, int block,
                                               int begin, int stride, int split) {
  constexpr int kOut = kGated ? kRows / 2 : kRows;  // columns of the cluster
  const int columns = kGated ? a.n / 2 : a.n;
  const int c0 = block * kOut;
  for (int i = begin; i < kOut * a.tokens; i += stride) {
    const int tok = i / kOut, c = i % kOut;
    if (c0 + c >= columns) continue;
    const auto sum = [&](int row) {
      const float* at = part + tok * (kRows + kSumPad) + row;
      if (split == 1) return *at;
      float v = 0.f;
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < split) v += ld_cluster_f32(map_to_cta(smem_u32(at), static_cast<uint32_t>(r)));
      return v;
    };
    float v;
    if constexpr (kGated) {
      const int row = c / 16 * 32 + c % 16;
      v = silu_times(sum(row), sum(row + 16));
    } else {
      v = sum(c);
    }
    const long long at = static_cast<long long>(tok) * columns + c0 + c;
    if (a.addend != nullptr) v += a.addend[at];
    if (a.f32_out)
      static_cast<float*>(a.out)[at] = v;
    else
      static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
  }
}

}  // namespace

}  // namespace w4a16
