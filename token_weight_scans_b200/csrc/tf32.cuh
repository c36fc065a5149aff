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

// Operand fragments of one warp: 16 rows x 8 of A(row, k), 8 of B(k, column) x 8 columns. kExact:
// the values are exact in tf32 (bf16 ones).
struct A16 { uint32_t hi[4], lo[4]; };
struct B8 { uint32_t hi[2], lo[2]; };
template <typename F>
__device__ __forceinline__ A16 load_a(F A) {
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  A16 a;
  split(A(g, t), a.hi[0], a.lo[0]);
  split(A(g + 8, t), a.hi[1], a.lo[1]);
  split(A(g, t + 4), a.hi[2], a.lo[2]);
  split(A(g + 8, t + 4), a.hi[3], a.lo[3]);
  return a;
}
template <bool kExact, typename F>
__device__ __forceinline__ B8 load_b(F B) {
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  B8 b;
  if (kExact) {
    b.hi[0] = __float_as_uint(B(t, g));
    b.hi[1] = __float_as_uint(B(t + 4, g));
  } else {
    split(B(t, g), b.hi[0], b.lo[0]);
    split(B(t + 4, g), b.hi[1], b.lo[1]);
  }
  return b;
}
// c += a b. c[0], c[1] are in row lane / 4 at columns 2 (lane % 4) and the next, c[2], c[3] eight
// rows below. The tensor core cuts off its sums where a float32 addition rounds, always towards
// zero, so that a long chain of them drifts: it sums the three products of one step alone, and
// they are added to c by float32 additions (the gradients 2.5e-7 off, 1.05e-6 in one chain; 495
// against 490 us for training B4 H8 T2048 d64).
template <bool kExactB>
__device__ __forceinline__ void mma3(float (&c)[4], const A16& a, const B8& b) {
  float p[4] = {0.f, 0.f, 0.f, 0.f};
  if (!kExactB) mma(p, a.hi, b.lo);
  mma(p, a.lo, b.hi);
  mma(p, a.hi, b.hi);
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] += p[e];
}

// One warp: c += A B over k0 <= k < k1 (whole eights).
template <bool kExactB, typename FA, typename FB>
__device__ __forceinline__ void tile(float (&c)[4], int k0, int k1, FA A, FB B) {
  float big[4] = {0.f, 0.f, 0.f, 0.f}, s0[4] = {0.f, 0.f, 0.f, 0.f};
  float s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = k0; k < k1; k += 8) {
    const A16 a = load_a([&](int r, int kk) { return A(r, k + kk); });
    const B8 b = load_b<kExactB>([&](int kk, int n) { return B(k + kk, n); });
    mma(big, a.hi, b.hi);
    if (!kExactB) mma(s0, a.hi, b.lo);
    mma(s1, a.lo, b.hi);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] += big[e] + (s0[e] + s1[e]);
}

}  // namespace tf32
}  // namespace gradlev
