// Tensor-core gated delta rule: few long scans in segments, and the order of the kernels.
//
// Within a segment the state after is affine in the state before, S_end = S_start M + L, with
// one 128 x 128 matrix M per (b, h, segment) that every row of S shares: the products of the
// chunks' maps. A first walk over all segments at once carries zero (which gives L) and, as
// one more slice of rows, the identity (which gives M); launch_combine runs the short serial
// recursion over the segments; the walk proper then starts every segment from its own state.
// Backward the same with dS_start = dS_end M^T + L', with the M of the forward.
//
// The first walk costs about as much again, so segments pay where the scans leave the GPU
// idle: B1 H16 T32768 d_v 256 has 32 CTAs of 512 chunks without them, and with four segments
// 144 and then 144 of 128 chunks. Measured there: forward with the last state 463 us for the
// first walk, 23 for the combination and 466 for the walk proper (the whole call 1299 us, 2108 in one
// walk); in training 319, 22 and 484, backward 241, 23 and 387 (2378 us, 3803 in one walk).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <atomic>

#include "delta_tc.h"
#include "sm100.cuh"

namespace gradlev {
namespace delta {
namespace tc {

namespace {

constexpr int kSMs = 148;
constexpr int kMinChunks = 12;   // per segment: below, the two extra kernels (30 us) cost more
constexpr int kMaxSeg = 16;
constexpr int kThreads = 256;

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

size_t state_bytes(const Dims& d, int nseg) {
  return up256(d.BH() * nseg * dvp(d) * 128 * sizeof(float));
}

constexpr int kLd = 132;         // row stride of M in shared memory: 16-byte rows, no bank conflicts
template <int kRows> constexpr size_t combine_smem() { return (2 * 128 + kRows) * kLd * sizeof(float); }

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (unsigned)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}

// kRows rows of one scan through its segments: out[s] = out[s -+ 1] M (M^T) + L. Thread: column
// c, kRows / 2 rows. BWD: from the last segment. The next segment's M lands while this one's is
// used (5 us a step; 12 us when it was read straight from memory).
template <bool BWD, int kRows>
__global__ void __launch_bounds__(kThreads) combine_kernel(Dims d, int nseg, const float* L,
                                                           const float* M, const float* S0,
                                                           const float* log_alpha, const bf16* dST,
                                                           float* out) {
  extern __shared__ __align__(16) float sm[];
  float* S = sm + 2 * 128 * kLd;  // [kRows][kLd]
  const int dv = dvp(d), nb = dv / kRows, bh = blockIdx.x / nb, r0 = (blockIdx.x - bh * nb) * kRows;
  const int c = threadIdx.x & 127, h = (threadIdx.x >> 7) * (kRows / 2);
  auto seg_at = [&](int i) { return (size_t)bh * nseg + (BWD ? nseg - 1 - i : i); };
  auto fetch = [&](int i) {
    if (i + 1 < nseg) {
      const float* m = M + seg_at(i) * 128 * 128;
      float* d = sm + (i & 1) * 128 * kLd;
      for (int j = threadIdx.x; j < 128 * 32; j += kThreads)
        copy16(d + (j >> 5) * kLd + 4 * (j & 31), m + 4 * j);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  const bool use_S0 = S0 && !(log_alpha[(size_t)bh * d.T] < kResetLog);
  float s[kRows / 2];
#pragma unroll
  for (int e = 0; e < kRows / 2; ++e) {
    const int r = r0 + h + e;  // the caller's states have no padding
    const bool ok = r < d.dv && c < d.dk;
    const size_t at = ((size_t)bh * d.dv + r) * d.dk + c;
    s[e] = !ok ? 0.f : BWD ? (dST ? __bfloat162float(dST[at]) : 0.f) : (use_S0 ? S0[at] : 0.f);
  }
  fetch(0);
  for (int i = 0; i < nseg; ++i) {
    const size_t sg = seg_at(i);
#pragma unroll
    for (int e = 0; e < kRows / 2; ++e) {
      out[(sg * dv + r0 + h + e) * 128 + c] = s[e];
      S[(h + e) * kLd + c] = s[e];
    }
    if (i + 1 == nseg) break;
    fetch(i + 1);
#pragma unroll
    for (int e = 0; e < kRows / 2; ++e) s[e] = L[(sg * dv + r0 + h + e) * 128 + c];
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const float* m = sm + (i & 1) * 128 * kLd;
#pragma unroll 4
    for (int k = 0; k < 128; k += 4) {
      const float4 mv = BWD ? *reinterpret_cast<const float4*>(m + c * kLd + k)
                            : make_float4(m[k * kLd + c], m[(k + 1) * kLd + c],
                                          m[(k + 2) * kLd + c], m[(k + 3) * kLd + c]);
#pragma unroll
      for (int e = 0; e < kRows / 2; ++e) {
        const float4 v = *reinterpret_cast<const float4*>(S + (h + e) * kLd + k);
        s[e] = fmaf(v.x, mv.x, s[e]);
        s[e] = fmaf(v.y, mv.y, s[e]);
        s[e] = fmaf(v.z, mv.z, s[e]);
        s[e] = fmaf(v.w, mv.w, s[e]);
      }
    }
    __syncthreads();
  }
}

template <bool BWD, int kRows>
cudaError_t combine(const Args& a, cudaStream_t st) {
  static std::atomic<uint64_t> set{0};  // devices whose opt-in is done
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!bit || !(set.load() & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(
        combine_kernel<BWD, kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        (int)combine_smem<kRows>());
    if (e != cudaSuccess) return e;
    set.fetch_or(bit);
  }
  const cudaError_t e = launch_after(
      launches_early(a.d, a.ST != nullptr), combine_kernel<BWD, kRows>, (unsigned)(a.d.BH() * (dvp(a.d) / kRows)), kThreads,
      combine_smem<kRows>(), st, a.d, a.seg.nseg, (const float*)a.loc, (const float*)a.M, a.S0,
      a.log_alpha, static_cast<const bf16*>(a.dST), a.init);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace

// The most segments whose CTAs still run at once, both in the first walk (the slices and the
// identity, all segments but one) and in the walk proper (and the last segment's identity).
SegPlan seg_plan(const Dims& d) {
  const long long BH = (long long)d.B * d.H, ns = dvp(d) / 128;
  const int N = chunks(d.T);
  for (int s = kMaxSeg; s >= 3; --s) {
    const int per = (N + s - 1) / s, nseg = (N + per - 1) / per;
    if (nseg >= 3 && per >= kMinChunks && BH * (ns + 1) * (nseg - 1) <= kSMs &&
        BH * (ns * nseg + 1) <= kSMs)
      return SegPlan{nseg, per};
  }
  return SegPlan{1, N};
}

size_t seg_bytes(const Dims& d, bool own_M) {
  const SegPlan s = seg_plan(d);
  if (s.nseg == 1) return 0;
  return 2 * state_bytes(d, s.nseg) + (own_M ? d.BH() * s.nseg * 128 * 128 * sizeof(float) : 0);
}

void set_segments(Args& a, char* at, float* M) {
  a.seg = seg_plan(a.d);
  if (a.seg.nseg == 1) return;
  a.loc = reinterpret_cast<float*>(at);
  a.init = reinterpret_cast<float*>(at + state_bytes(a.d, a.seg.nseg));
  a.M = M ? M : reinterpret_cast<float*>(at + 2 * state_bytes(a.d, a.seg.nseg));
}

cudaError_t launch_combine(const Args& a, bool backward, cudaStream_t st) {
  // One CTA per SM (two M tiles): 16 rows each (5 us a step) while those run at once, 32 (7 us)
  // beyond.
  if (a.d.BH() * (dvp(a.d) / 16) <= kSMs)
    return backward ? combine<true, 16>(a, st) : combine<false, 16>(a, st);
  return backward ? combine<true, 32>(a, st) : combine<false, 32>(a, st);
}

// ---------------------------------------------------------------- the kernels in order
static cudaError_t walk(const Args& a, bool backward, bool last_state, cudaStream_t st) {
  if (a.seg.nseg > 1) {
    cudaError_t e = launch_walk(a, backward, last_state, true, !backward, st);
    if (e == cudaSuccess) e = launch_combine(a, backward, st);
    if (e != cudaSuccess) return e;
  }
  return launch_walk(a, backward, last_state, false, !backward || a.seg.nseg > 1, st);
}

cudaError_t run_fwd(const Args& a, cudaStream_t st) {
  const bool last_state = a.ST != nullptr;
  const cudaError_t e = launch_prep(a, last_state, st);
  return e != cudaSuccess ? e : walk(a, false, last_state, st);
}

cudaError_t run_bwd(const Args& a, cudaStream_t st) {
  const cudaError_t e = walk(a, true, false, st);
  return e != cudaSuccess ? e : launch_grad(a, st);
}

// ---------------------------------------------------------------- buffers
static bf16* take(char*& at, size_t elems) {
  bf16* p = reinterpret_cast<bf16*>(at);
  at += up256(elems * sizeof(bf16));
  return p;
}
static size_t gate_bytes(const Dims& d) {
  return up256(d.BH() * chunks(d.T) * sizeof(GateBlock));
}
size_t token_rows_bytes(const Dims& d) {
  return up256(d.BH() * chunks(d.T) * 2 * dvp(d) * C * sizeof(bf16));
}
// one of struct Mats
static size_t mat_bytes(const Dims& d) { return up256(d.BH() * chunks(d.T) * C * 128 * sizeof(bf16)); }

Saved saved_at(char* base, const Dims& d) {
  const size_t rows = d.BH() * chunks(d.T);
  char* at = base;
  Saved s;
  s.S = take(at, rows * dvp(d) * 128);
  s.D = take(at, rows * 2 * dvp(d) * C);
  for (bf16** m : {&s.Kw, &s.Wq, &s.Wq2, &s.Pv}) *m = take(at, rows * C * 128);
  s.gates = reinterpret_cast<float*>(at);
  s.M = reinterpret_cast<float*>(at + gate_bytes(d));
  return s;
}

size_t saved_bytes(const Dims& d) {
  const size_t rows = d.BH() * chunks(d.T);
  const int nseg = seg_plan(d).nseg;
  return up256(rows * dvp(d) * 256) + token_rows_bytes(d) + 4 * mat_bytes(d) + gate_bytes(d) +
         (nseg > 1 ? d.BH() * nseg * 128 * 128 * sizeof(float) : 0);
}

// With checkpoints Kw, Wq, Pv and the gates are among them, and T0 is needed for D.
Mats mats_at(char* base, const Dims& d, bool saved) {
  const size_t n = d.BH() * chunks(d.T) * C * 128;
  char* at = base;
  Mats m;
  m.Kw2 = take(at, n);
  m.Kw3 = take(at, n);
  if (saved) {
    m.T0 = take(at, n);
    return m;
  }
  for (bf16** x : {&m.Kw, &m.Wq, &m.Pv}) *x = take(at, n);
  m.gates = reinterpret_cast<float*>(at);
  return m;
}

size_t fwd_scratch_bytes(const Dims& d) {  // the segments' buffers come last
  return 5 * mat_bytes(d) + gate_bytes(d) + seg_bytes(d, true);
}

size_t bwd_scratch_bytes(const Dims& d) {  // E, dS, the segments' buffers
  return token_rows_bytes(d) + up256(d.BH() * chunks(d.T) * dvp(d) * 256) + seg_bytes(d, false);
}

}  // namespace tc
}  // namespace delta
}  // namespace gradlev
