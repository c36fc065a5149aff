// The gated delta rule on CUDA cores (float32 arithmetic): every shape and dtype the
// tensor-core kernels do not take. The formulas are in delta.h.
//
// Four kernels. The chunk-local part (Z, P) and the gradients of q, k and the gates
// need no order among the chunks and run one CTA per chunk; only the two state
// recurrences walk the chunks in order. The rows of S (and of dS) evolve
// independently given K, so a walk is cut into slices of kRows rows, one CTA each.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "delta.h"

namespace gradlev {
namespace delta {
namespace ffma {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 16;     // state rows per CTA of a walk
__host__ __device__ constexpr int slices(int dv) { return (dv + kRows - 1) / kRows; }
constexpr int LD = C + 1;     // row stride of a C x C matrix in shared memory

// Gates of one chunk. The running sum is kept in double: over a chunk of strong decays L
// reaches -32 * 87, where a float32 sum would leave 1e-4 in the differences.
struct Gates {
  double L[C];
  float beta[C], G[C], w[C];
  int seg[C];
  float GC;
};

// One warp fills the gates of tokens [t0, t0 + C) (beta = 0, a = 1 past T).
__device__ void load_gates(Gates& g, const float* beta, const float* log_alpha, size_t row, int t0,
                           int T) {
  const int lane = threadIdx.x & 31;
  const bool in = t0 + lane < T;
  const float la = in ? log_alpha[row + t0 + lane] : 0.f;
  const float be = in ? beta[row + t0 + lane] : 0.f;
  const bool reset = la < kResetLog;
  double L = reset ? 0.0 : (double)la;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(0xffffffffu, L, o);
    if (lane >= o) L += u;
  }
  const unsigned mask = __ballot_sync(0xffffffffu, reset);
  const int seg = __popc(mask & (0xffffffffu >> (31 - lane)));
  const double Lend = __shfl_sync(0xffffffffu, L, 31);
  const int send = __popc(mask);
  g.L[lane] = L;
  g.beta[lane] = be;
  g.seg[lane] = seg;
  g.G[lane] = seg == 0 ? expf((float)L) : 0.f;
  g.w[lane] = seg == send ? expf((float)(Lend - L)) : 0.f;
  if (lane == 0) g.GC = send == 0 ? expf((float)Lend) : 0.f;
}

__device__ __forceinline__ float decay(const Gates& g, int i, int j) {  // M_ij, j <= i
  return g.seg[i] == g.seg[j] ? expf((float)(g.L[i] - g.L[j])) : 0.f;
}

// Rows [t0, t0 + C) x columns [c0, c0 + n) of a [T][ld] matrix into dst[C][ldd], zero past T.
template <typename Tio>
__device__ void load_tile(float* dst, int ldd, const Tio* src, size_t ld, int t0, int T, int c0,
                          int n) {
  for (int i = threadIdx.x; i < C * n; i += kThreads) {
    const int r = i / n, c = i - r * n;
    dst[r * ldd + c] = t0 + r < T ? to_f32(src[(size_t)(t0 + r) * ld + c0 + c]) : 0.f;
  }
}

__device__ __forceinline__ float dot4(const float4& a, const float4& b, float s) {
  s = fmaf(a.x, b.x, s);
  s = fmaf(a.y, b.y, s);
  s = fmaf(a.z, b.z, s);
  return fmaf(a.w, b.w, s);
}
__device__ __forceinline__ float4 at4(const float* p) { return *reinterpret_cast<const float4*>(p); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__host__ __device__ constexpr int pad4(int n) { return n + 4; }  // row stride: 16-byte rows, no bank conflicts

// ------------------------------------------------------------------ Z and P of every chunk
template <typename Tio>
__global__ void __launch_bounds__(kThreads) prep_kernel(Args a) {
  extern __shared__ __align__(16) float sm[];
  __shared__ Gates g;
  __shared__ float A[C * LD], Zs[C * LD];
  const Dims& d = a.d;
  const int N = chunks(d.T), bh = blockIdx.x / N, n = blockIdx.x - bh * N;
  const int b = bh / d.H, h = bh - b * d.H;
  const size_t kh = (size_t)b * d.Hk + h / (d.H / d.Hk);
  const int ld = pad4(d.dk), t0 = n * C;
  float *K = sm, *Q = sm + C * ld;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) load_gates(g, a.beta, a.log_alpha, (size_t)bh * d.T, t0, d.T);
  load_tile(K, ld, static_cast<const Tio*>(a.k) + kh * d.T * d.dk, d.dk, t0, d.T, 0, d.dk);
  load_tile(Q, ld, static_cast<const Tio*>(a.q) + kh * d.T * d.dk, d.dk, t0, d.T, 0, d.dk);
  __syncthreads();
  const size_t cc = ((size_t)bh * N + n) * C * C;
  for (int i = warp; i < C; i += kWarps) {
    float kk = 0.f, qk = 0.f;
    for (int c = 0; c < d.dk; c += 4) {
      const float4 kj = at4(K + lane * ld + c);
      kk = dot4(at4(K + i * ld + c), kj, kk);
      qk = dot4(at4(Q + i * ld + c), kj, qk);
    }
    const float m = lane <= i ? decay(g, i, lane) : 0.f;
    A[i * LD + lane] = lane < i ? m * kk : 0.f;
    a.sv.P[cc + i * C + lane] = lane <= i ? a.scale * m * qk : 0.f;
  }
  __syncthreads();
  // Z_ij = A_ij - sum_{j<m<i} A_im beta_m Z_mj: lane j owns column j, row by row. A lane
  // reads back only what it wrote itself.
  if (warp == 0) {
    for (int i = 0; i < C; ++i) {
      float z = A[i * LD + lane];
      for (int m = 0; m < i; ++m) z = fmaf(-A[i * LD + m] * g.beta[m], m > lane ? Zs[m * LD + lane] : 0.f, z);
      Zs[i * LD + lane] = z;
      a.sv.Z[cc + i * C + lane] = z;
    }
  }
}

// ------------------------------------------------------------------ forward walk
template <typename Tio>
__global__ void __launch_bounds__(kThreads) fwd_kernel(Args a) {
  extern __shared__ __align__(16) float sm[];
  __shared__ Gates g;
  __shared__ float Z[C * LD], P[C * LD];
  __shared__ __align__(16) float R[C * kRows], D[C * kRows];  // read as float4
  const Dims& d = a.d;
  const int N = chunks(d.T), ns = slices(d.dv), bh = blockIdx.x / ns;
  const int n0 = (blockIdx.x - bh * ns) * kRows;
  const int rows = min(kRows, d.dv - n0);
  const int b = bh / d.H, h = bh - b * d.H;
  const size_t kh = (size_t)b * d.Hk + h / (d.H / d.Hk);
  const int ld = pad4(d.dk);
  float *K = sm, *Q = K + C * ld, *S = Q + C * ld;  // S [kRows][ld]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = 2 * warp;  // this thread: token `lane`, rows r0 and r0 + 1
  for (int i = tid; i < kRows * d.dk; i += kThreads) {
    const int r = i / d.dk, c = i - r * d.dk;
    S[r * ld + c] = a.S0 && r < rows ? a.S0[((size_t)bh * d.dv + n0 + r) * d.dk + c] : 0.f;
  }
  for (int n = 0; n < N; ++n) {
    const int t0 = n * C;
    __syncthreads();
    if (warp == 0) load_gates(g, a.beta, a.log_alpha, (size_t)bh * d.T, t0, d.T);
    load_tile(K, ld, static_cast<const Tio*>(a.k) + kh * d.T * d.dk, d.dk, t0, d.T, 0, d.dk);
    load_tile(Q, ld, static_cast<const Tio*>(a.q) + kh * d.T * d.dk, d.dk, t0, d.T, 0, d.dk);
    for (int i = tid; i < C * kRows; i += kThreads) {
      const int t = i / kRows, r = i - t * kRows;
      R[i] = t0 + t < d.T && r < rows
                 ? to_f32(static_cast<const Tio*>(a.v)[((size_t)bh * d.T + t0 + t) * d.dv + n0 + r])
                 : 0.f;
    }
    const size_t cc = ((size_t)bh * N + n) * C * C;
    for (int i = tid; i < C * C; i += kThreads) {
      Z[(i / C) * LD + i % C] = a.sv.Z[cc + i];
      P[(i / C) * LD + i % C] = a.sv.P[cc + i];
    }
    if (a.sv.S) {
      float* out = a.sv.S + (((size_t)bh * N + n) * d.dv + n0) * d.dk;
      for (int i = tid; i < rows * d.dk; i += kThreads) out[i] = S[(i / d.dk) * ld + i % d.dk];
    }
    __syncthreads();
    // K S^T and Q S^T
    float x0 = 0.f, x1 = 0.f, y0 = 0.f, y1 = 0.f;
    for (int c = 0; c < d.dk; c += 4) {
      const float4 kv = at4(K + lane * ld + c), qv = at4(Q + lane * ld + c);
      const float4 s0 = at4(S + r0 * ld + c), s1 = at4(S + (r0 + 1) * ld + c);
      x0 = dot4(kv, s0, x0);
      x1 = dot4(kv, s1, x1);
      y0 = dot4(qv, s0, y0);
      y1 = dot4(qv, s1, y1);
    }
    const float Gi = g.G[lane];
    x0 = R[lane * kRows + r0] - Gi * x0;
    x1 = R[lane * kRows + r0 + 1] - Gi * x1;
    __syncwarp();  // a warp's rows of R are its own
    R[lane * kRows + r0] = x0;
    R[lane * kRows + r0 + 1] = x1;
    __syncwarp();
    for (int m = 0; m < C; ++m) {
      const float z = -Z[lane * LD + m] * g.beta[m];
      x0 = fmaf(z, R[m * kRows + r0], x0);
      x1 = fmaf(z, R[m * kRows + r0 + 1], x1);
    }
    D[lane * kRows + r0] = x0;
    D[lane * kRows + r0 + 1] = x1;
    __syncwarp();
    y0 *= a.scale * Gi;
    y1 *= a.scale * Gi;
    for (int m = 0; m < C; ++m) {
      const float p = P[lane * LD + m] * g.beta[m];
      y0 = fmaf(p, D[m * kRows + r0], y0);
      y1 = fmaf(p, D[m * kRows + r0 + 1], y1);
    }
    __syncwarp();
    R[lane * kRows + r0] = y0;
    R[lane * kRows + r0 + 1] = y1;
    __syncthreads();
    for (int i = tid; i < C * kRows; i += kThreads) {
      const int t = i / kRows, r = i - t * kRows;
      if (t0 + t < d.T && r < rows) {
        const size_t at = ((size_t)bh * d.T + t0 + t) * d.dv + n0 + r;
        if (a.y) static_cast<Tio*>(a.y)[at] = from_f32<Tio>(R[i]);
        if (a.sv.D) a.sv.D[at] = D[i];
      }
    }
    // S <- G_C S + D^T diag(beta w) K
    const float GC = g.GC;
    for (int i = tid; i < kRows / 4 * d.dk; i += kThreads) {
      const int rq = i / d.dk, c = i - rq * d.dk;
      float s[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = GC * S[(4 * rq + e) * ld + c];
      for (int m = 0; m < C; ++m) {
        const float kv = K[m * ld + c] * (g.beta[m] * g.w[m]);
        const float4 dd = at4(D + m * kRows + 4 * rq);
        s[0] = fmaf(dd.x, kv, s[0]);
        s[1] = fmaf(dd.y, kv, s[1]);
        s[2] = fmaf(dd.z, kv, s[2]);
        s[3] = fmaf(dd.w, kv, s[3]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) S[(4 * rq + e) * ld + c] = s[e];
    }
  }
  __syncthreads();
  if (a.ST)
    for (int i = tid; i < rows * d.dk; i += kThreads)
      a.ST[((size_t)bh * d.dv + n0) * d.dk + i] = S[(i / d.dk) * ld + i % d.dk];
}

// ------------------------------------------------------------------ backward walk
template <typename Tio>
__global__ void __launch_bounds__(kThreads) bwd_kernel(Args a) {
  extern __shared__ __align__(16) float sm[];
  __shared__ Gates g;
  __shared__ float Z[C * LD], P[C * LD];
  __shared__ __align__(16) float R[C * kRows], F[C * kRows];  // read as float4
  const Dims& d = a.d;
  const int N = chunks(d.T), ns = slices(d.dv), bh = blockIdx.x / ns;
  const int n0 = (blockIdx.x - bh * ns) * kRows;
  const int rows = min(kRows, d.dv - n0);
  const int b = bh / d.H, h = bh - b * d.H;
  const size_t kh = (size_t)b * d.Hk + h / (d.H / d.Hk);
  const int ld = pad4(d.dk);
  float *K = sm, *Q = K + C * ld, *S = Q + C * ld;  // S [kRows][ld]: dS
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = 2 * warp;
  for (int i = tid; i < kRows * d.dk; i += kThreads) {
    const int r = i / d.dk, c = i - r * d.dk;
    S[r * ld + c] =
        a.dST && r < rows
            ? to_f32(static_cast<const Tio*>(a.dST)[((size_t)bh * d.dv + n0 + r) * d.dk + c])
            : 0.f;
  }
  for (int n = N - 1; n >= 0; --n) {
    const int t0 = n * C;
    __syncthreads();
    if (warp == 0) load_gates(g, a.beta, a.log_alpha, (size_t)bh * d.T, t0, d.T);
    load_tile(K, ld, static_cast<const Tio*>(a.k) + kh * d.T * d.dk, d.dk, t0, d.T, 0, d.dk);
    load_tile(Q, ld, static_cast<const Tio*>(a.q) + kh * d.T * d.dk, d.dk, t0, d.T, 0, d.dk);
    for (int i = tid; i < C * kRows; i += kThreads) {
      const int t = i / kRows, r = i - t * kRows;
      R[i] = t0 + t < d.T && r < rows
                 ? to_f32(static_cast<const Tio*>(a.dy)[((size_t)bh * d.T + t0 + t) * d.dv + n0 + r])
                 : 0.f;
    }
    const size_t cc = ((size_t)bh * N + n) * C * C;
    for (int i = tid; i < C * C; i += kThreads) {
      Z[(i / C) * LD + i % C] = a.sv.Z[cc + i];
      P[(i / C) * LD + i % C] = a.sv.P[cc + i];
    }
    {
      float* out = a.dS + (((size_t)bh * N + n) * d.dv + n0) * d.dk;
      for (int i = tid; i < rows * d.dk; i += kThreads) out[i] = S[(i / d.dk) * ld + i % d.dk];
    }
    __syncthreads();
    float x0 = 0.f, x1 = 0.f;
    for (int c = 0; c < d.dk; c += 4) {
      const float4 kv = at4(K + lane * ld + c);
      x0 = dot4(kv, at4(S + r0 * ld + c), x0);
      x1 = dot4(kv, at4(S + (r0 + 1) * ld + c), x1);
    }
    x0 *= g.w[lane];
    x1 *= g.w[lane];
    for (int m = 0; m < C; ++m) {  // P^T dY
      const float p = P[m * LD + lane];
      x0 = fmaf(p, R[m * kRows + r0], x0);
      x1 = fmaf(p, R[m * kRows + r0 + 1], x1);
    }
    F[lane * kRows + r0] = x0;
    F[lane * kRows + r0 + 1] = x1;
    __syncwarp();
    for (int m = 0; m < C; ++m) {  // - Z^T diag(beta) F
      const float z = -Z[m * LD + lane] * g.beta[m];
      x0 = fmaf(z, F[m * kRows + r0], x0);
      x1 = fmaf(z, F[m * kRows + r0 + 1], x1);
    }
    __syncwarp();
    F[lane * kRows + r0] = x0;  // E
    F[lane * kRows + r0 + 1] = x1;
    __syncthreads();
    for (int i = tid; i < C * kRows; i += kThreads) {
      const int t = i / kRows, r = i - t * kRows;
      if (t0 + t < d.T && r < rows) {
        const size_t at = ((size_t)bh * d.T + t0 + t) * d.dv + n0 + r;
        a.E[at] = F[i];
        static_cast<Tio*>(a.dv_)[at] = from_f32<Tio>(g.beta[t] * F[i]);
      }
    }
    const float GC = g.GC;
    for (int i = tid; i < kRows / 4 * d.dk; i += kThreads) {
      const int rq = i / d.dk, c = i - rq * d.dk;
      float s[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = GC * S[(4 * rq + e) * ld + c];
      for (int m = 0; m < C; ++m) {
        const float qv = Q[m * ld + c] * (a.scale * g.G[m]);
        const float kv = -K[m * ld + c] * (g.beta[m] * g.G[m]);
        const float4 oo = at4(R + m * kRows + 4 * rq), ee = at4(F + m * kRows + 4 * rq);
        s[0] = fmaf(ee.x, kv, fmaf(oo.x, qv, s[0]));
        s[1] = fmaf(ee.y, kv, fmaf(oo.y, qv, s[1]));
        s[2] = fmaf(ee.z, kv, fmaf(oo.z, qv, s[2]));
        s[3] = fmaf(ee.w, kv, fmaf(oo.w, qv, s[3]));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) S[(4 * rq + e) * ld + c] = s[e];
    }
  }
  __syncthreads();
  if (a.dS0)
    for (int i = tid; i < rows * d.dk; i += kThreads)
      static_cast<Tio*>(a.dS0)[((size_t)bh * d.dv + n0) * d.dk + i] =
          from_f32<Tio>(S[(i / d.dk) * ld + i % d.dk]);
}

// ------------------------------------------------------------------ gradients of q, k, gates
// One CTA per (chunk, key head). A warp owns 4 tokens and every column, so a token's dot
// products end in a warp sum; the value heads that share the key head are walked in order
// and add up in registers.
template <typename Tio, int NJ>  // NJ: 32-column groups that cover dk
__global__ void __launch_bounds__(kThreads) grad_kernel(Args a) {
  extern __shared__ __align__(16) float sm[];
  __shared__ Gates g;
  __shared__ float X[C * LD], Y[C * LD], W[C * LD];  // W: X q.k - Y k.k
  __shared__ float dLx[C], dLz[C], red[kWarps];
  const Dims& d = a.d;
  const int N = chunks(d.T), n = blockIdx.x % N, t0 = n * C;
  const size_t kh = blockIdx.x / N;
  const int b = kh / d.Hk, hk = kh - (size_t)b * d.Hk, grp = d.H / d.Hk;
  const int ld = pad4(d.dk), lv = pad4(d.dv);
  float *K = sm, *Q = K + C * ld, *O = Q + C * ld, *D = O + C * lv, *E = D + C * lv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, i0 = 4 * warp;
  static_assert(4 * kWarps == C, "a warp owns 4 tokens");
  load_tile(K, ld, static_cast<const Tio*>(a.k) + kh * d.T * d.dk, d.dk, t0, d.T, 0, d.dk);
  load_tile(Q, ld, static_cast<const Tio*>(a.q) + kh * d.T * d.dk, d.dk, t0, d.T, 0, d.dk);
  __syncthreads();
  float kk[4], qk[4];  // k_i.k_j, q_i.k_j of this warp's tokens i, j = lane
#pragma unroll
  for (int e = 0; e < 4; ++e) kk[e] = qk[e] = 0.f;
  for (int c = 0; c < d.dk; c += 4) {
    const float4 kj = at4(K + lane * ld + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      kk[e] = dot4(at4(K + (i0 + e) * ld + c), kj, kk[e]);
      qk[e] = dot4(at4(Q + (i0 + e) * ld + c), kj, qk[e]);
    }
  }
  float aq[4][NJ], ak[4][NJ];
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int j = 0; j < NJ; ++j) aq[e][j] = ak[e][j] = 0.f;

  for (int hh = 0; hh < grp; ++hh) {
    const size_t bh = (size_t)b * d.H + hk * grp + hh;
    __syncthreads();
    if (warp == 0) load_gates(g, a.beta, a.log_alpha, bh * d.T, t0, d.T);
    load_tile(O, lv, static_cast<const Tio*>(a.dy) + bh * d.T * d.dv, d.dv, t0, d.T, 0, d.dv);
    load_tile(D, lv, a.sv.D + bh * d.T * d.dv, d.dv, t0, d.T, 0, d.dv);
    load_tile(E, lv, a.E + bh * d.T * d.dv, d.dv, t0, d.T, 0, d.dv);
    __syncthreads();
    const float* S = a.sv.S + (bh * N + n) * d.dv * d.dk;
    const float* dS = a.dS + (bh * N + n) * d.dv * d.dk;
    {  // X, Y, their part of dlog_alpha, dbeta
      float f[4], ed[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = ed[e] = 0.f;
      for (int c = 0; c < d.dv; c += 4) {
        const float4 dj = at4(D + lane * lv + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[e] = dot4(at4(O + (i0 + e) * lv + c), dj, f[e]);
          ed[e] = dot4(at4(E + (i0 + e) * lv + c), dj, ed[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + e;
        const float m = lane <= i ? decay(g, i, lane) * g.beta[lane] : 0.f;
        const float x = a.scale * m * f[e], y = lane < i ? m * g.beta[i] * ed[e] : 0.f;
        X[i * LD + lane] = x;
        Y[i * LD + lane] = y;
        W[i * LD + lane] = lane < i ? x * qk[e] - y * kk[e] : 0.f;
        const float db = __shfl_sync(0xffffffffu, ed[e], i);
        if (lane == 0 && t0 + i < d.T)
          static_cast<Tio*>(a.dbeta)[bh * d.T + t0 + i] = from_f32<Tio>(db);
      }
    }
    // dY S, E S, D dS: columns lane + 32 j
    float t[4][NJ], u[4][NJ], z[4][NJ];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < NJ; ++j) t[e][j] = u[e][j] = z[e][j] = 0.f;
    float ss = 0.f;
    for (int v = 0; v < d.dv; ++v) {
      float o[4], ee[4], dd[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[e] = O[(i0 + e) * lv + v];
        ee[e] = E[(i0 + e) * lv + v];
        dd[e] = D[(i0 + e) * lv + v];
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int c = lane + 32 * j;
        const float s = c < d.dk ? S[(size_t)v * d.dk + c] : 0.f;
        const float ds = c < d.dk ? dS[(size_t)v * d.dk + c] : 0.f;
        if ((v & (kWarps - 1)) == warp) ss = fmaf(s, ds, ss);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          t[e][j] = fmaf(o[e], s, t[e][j]);
          u[e][j] = fmaf(ee[e], s, u[e][j]);
          z[e][j] = fmaf(dd[e], ds, z[e][j]);
        }
      }
    }
    ss = warp_sum(ss);
    if (lane == 0) red[warp] = ss;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + e;
      const float cq = a.scale * g.G[i], ck = g.beta[i] * g.G[i], cz = g.beta[i] * g.w[i];
      float x = 0.f, zz = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int c = lane + 32 * j;
        const float qv = c < d.dk ? Q[i * ld + c] : 0.f, kv = c < d.dk ? K[i * ld + c] : 0.f;
        x += cq * t[e][j] * qv - ck * u[e][j] * kv;
        zz += cz * z[e][j] * kv;
        aq[e][j] += cq * t[e][j];
        ak[e][j] += cz * z[e][j] - ck * u[e][j];
      }
      x = warp_sum(x);
      zz = warp_sum(zz);
      if (lane == 0) {
        dLx[i] = x;
        dLz[i] = zz;
      }
    }
    __syncthreads();
    for (int m = 0; m < C; ++m) {
      float x[4], xt[4], yy[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = X[(i0 + e) * LD + m];
        xt[e] = X[m * LD + i0 + e];
        yy[e] = Y[(i0 + e) * LD + m] + Y[m * LD + i0 + e];
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int c = lane + 32 * j;
        const float qv = c < d.dk ? Q[m * ld + c] : 0.f, kv = c < d.dk ? K[m * ld + c] : 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          aq[e][j] = fmaf(x[e], kv, aq[e][j]);
          ak[e][j] = fmaf(xt[e], qv, fmaf(-yy[e], kv, ak[e][j]));
        }
      }
    }
    if (warp == 0) {
      // token `lane`: the pairs (i >= t > j) by the running sum of column sums - row sums
      float rc = 0.f;
      for (int m = 0; m < C; ++m) rc += W[lane * LD + m] - W[m * LD + lane];
      float x = dLx[lane] + rc, zz = dLz[lane];
      float acc = zz;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {  // suffix sum of x, prefix sum of z
        const float u1 = __shfl_down_sync(0xffffffffu, x, o);
        const float u2 = __shfl_up_sync(0xffffffffu, acc, o);
        if (lane + o < 32) x += u1;
        if (lane >= o) acc += u2;
      }
      float gg = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) gg += red[w];
      if (t0 + lane < d.T) {
        const bool reset = a.log_alpha[bh * d.T + t0 + lane] < kResetLog;
        static_cast<Tio*>(a.dlog_alpha)[bh * d.T + t0 + lane] =
            from_f32<Tio>(reset ? 0.f : x + (acc - zz) + g.GC * gg);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (t0 + i0 + e >= d.T) break;
    const size_t row = (kh * d.T + t0 + i0 + e) * d.dk;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int c = lane + 32 * j;
      if (c < d.dk) {
        static_cast<Tio*>(a.dq)[row + c] = from_f32<Tio>(aq[e][j]);
        static_cast<Tio*>(a.dk_)[row + c] = from_f32<Tio>(ak[e][j]);
      }
    }
  }
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// The 48 KB that need no opt-in hold the static arrays too.
template <typename F>
cudaError_t set_smem(F f, size_t bytes) {
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename Tio, int NJ>
cudaError_t launch_grad(const Args& a, cudaStream_t st) {
  const size_t smem =
      (size_t)C * (2 * pad4(a.d.dk) + 3 * pad4(a.d.dv)) * sizeof(float);
  const cudaError_t e = set_smem(grad_kernel<Tio, NJ>, smem);
  if (e != cudaSuccess) return e;
  grad_kernel<Tio, NJ><<<chunks(a.d.T) * a.d.B * a.d.Hk, kThreads, smem, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename Tio>
cudaError_t fwd_t(const Args& a, cudaStream_t st) {
  const Dims& d = a.d;
  const size_t sp = (size_t)2 * C * pad4(d.dk) * sizeof(float);
  cudaError_t e = set_smem(prep_kernel<Tio>, sp);
  if (e != cudaSuccess) return e;
  prep_kernel<Tio><<<chunks(d.T) * d.B * d.H, kThreads, sp, st>>>(a);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const size_t sf = (size_t)(2 * C + kRows) * pad4(d.dk) * sizeof(float);
  if ((e = set_smem(fwd_kernel<Tio>, sf)) != cudaSuccess) return e;
  fwd_kernel<Tio><<<slices(d.dv) * d.B * d.H, kThreads, sf, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename Tio>
cudaError_t bwd_t(const Args& a, cudaStream_t st) {
  const Dims& d = a.d;
  const size_t sf = (size_t)(2 * C + kRows) * pad4(d.dk) * sizeof(float);
  cudaError_t e = set_smem(bwd_kernel<Tio>, sf);
  if (e != cudaSuccess) return e;
  bwd_kernel<Tio><<<slices(d.dv) * d.B * d.H, kThreads, sf, st>>>(a);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (d.dk <= 64) return launch_grad<Tio, 2>(a, st);
  if (d.dk <= 128) return launch_grad<Tio, 4>(a, st);
  return launch_grad<Tio, 8>(a, st);
}

}  // namespace

size_t saved_bytes(const Dims& d, bool states) {
  const size_t N = chunks(d.T), cc = up256(d.BH() * N * C * C * sizeof(float));
  size_t n = 2 * cc;
  if (states)
    n += up256(d.BH() * N * d.dv * d.dk * sizeof(float)) +
         up256(d.BH() * (size_t)d.T * d.dv * sizeof(float));
  return n;
}

Saved saved_at(char* base, const Dims& d, bool states) {
  const size_t N = chunks(d.T), cc = up256(d.BH() * N * C * C * sizeof(float));
  Saved s{};
  s.Z = reinterpret_cast<float*>(base);
  s.P = reinterpret_cast<float*>(base + cc);
  if (states) {
    s.S = reinterpret_cast<float*>(base + 2 * cc);
    s.D = reinterpret_cast<float*>(base + 2 * cc +
                                   up256(d.BH() * N * d.dv * d.dk * sizeof(float)));
  }
  return s;
}

cudaError_t run_fwd(const Args& a, cudaStream_t st) {
  return a.d.bf16 ? fwd_t<__nv_bfloat16>(a, st) : fwd_t<float>(a, st);
}

cudaError_t run_bwd(const Args& a, cudaStream_t st) {
  return a.d.bf16 ? bwd_t<__nv_bfloat16>(a, st) : bwd_t<float>(a, st);
}

}  // namespace ffma
}  // namespace delta
}  // namespace gradlev
