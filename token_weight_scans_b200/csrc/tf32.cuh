// Products of float32 matrices by warp-wide tf32 instructions, for tiles too small to fill
// tcgen05.mma. An operand is split into two tf32 parts, x = hi + lo with |lo| <= 2^-11 |x|, and
// the product is hi hi + hi lo + lo hi: off by 2^-21 of |a| |b|, where one part each would be off
// by 2^-11. Against float32 FMAs it saves the reads of shared memory: a fragment's element is
// read once for 8 or 16 products.
#pragma once

#include <stdint.h>

namespace gradlev {
namespace tf32 {

// tf32 keeps 10 bits behind the point: hi rounds to nearest by an integer addition, lo is cut
// (2^-10 of 2^-11). Conversion instructions would do the same at a fraction of the rate.
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
               "{%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// One warp: c += A B over k0 <= k < k1 (whole eights), A(row, k) for 16 rows, B(k, column) for 8
// columns. c[0], c[1] are in row lane / 4 at columns 2 (lane % 4) and the next, c[2], c[3] eight
// rows below. kExactB: B is exact in tf32 (bf16 values).
template <bool kExactB, typename FA, typename FB>
__device__ __forceinline__ void tile(float (&c)[4], int k0, int k1, FA A, FB B) {
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  float big[4] = {0.f, 0.f, 0.f, 0.f}, s0[4] = {0.f, 0.f, 0.f, 0.f};
  float s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = k0; k < k1; k += 8) {
    uint32_t ah[4], al[4], bh[2], bl[2];
    split(A(g, k + t), ah[0], al[0]);
    split(A(g + 8, k + t), ah[1], al[1]);
    split(A(g, k + t + 4), ah[2], al[2]);
    split(A(g + 8, k + t + 4), ah[3], al[3]);
    if (kExactB) {
      bh[0] = __float_as_uint(B(k + t, g));
      bh[1] = __float_as_uint(B(k + t + 4, g));
    } else {
      split(B(k + t, g), bh[0], bl[0]);
      split(B(k + t + 4, g), bh[1], bl[1]);
    }
    mma(big, ah, bh);
    if (!kExactB) mma(s0, ah, bl);
    mma(s1, al, bh);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] += big[e] + (s0[e] + s1[e]);
}

}  // namespace tf32
}  // namespace gradlev
