// The gated delta rule in float32: every shape and dtype that the tcgen05 kernels do not take.
// The formulas are in delta.h.
//
// Four kernels. The chunk-local part (Z, P) and the gradients of q, k and the gates
// need no order among the chunks and run one CTA per chunk; only the two state
// recurrences walk the chunks in order. All products are warp tiles (mma.sync) of operands split
// into two tf32 each (tf32.cuh), whose sums are float32 additions: outputs are 2 to 4e-7 off, as
// with FMAs, which waited for shared memory and took half as long again. Sums, states and the
// chunk's triangular systems are float32. The rows of S (and of dS) evolve
// independently given K, so a walk is cut into slices of kRows rows, one CTA each.
//
// Measured (B4 H8 T2048 d 64): Z and P 36 us, walks 147 and 143 us (239 and 219 us with FMAs),
// gradients 169 us (235 us). A walk has 128 CTAs of one chain each, 2.2 us a chunk: four
// products in a row at 8 warps per SM (44 % of the issue slots). The gradients' kernel has 16
// warps per SM at 45 %: splitting operands is most of its instructions.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "delta.h"
#include "tf32.cuh"

namespace gradlev {
namespace delta {
namespace ffma {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 16;     // state rows per CTA of a walk
__host__ __device__ constexpr int slices(int dv) { return (dv + kRows - 1) / kRows; }
// row strides of a C x C matrix in shared memory: read by columns; by rows and in tiles
constexpr int LD = C + 1, LZ = C + 4;

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

__device__ __forceinline__ float dot4(const float4& a, const float4& b, float s) {
  s = fmaf(a.x, b.x, s);
  s = fmaf(a.y, b.y, s);
  s = fmaf(a.z, b.z, s);
  return fmaf(a.w, b.w, s);
}
__device__ __forceinline__ float4 at4(const float* p) { return *reinterpret_cast<const float4*>(p); }

__device__ __forceinline__ float4 at4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

// Rows [t0, t0 + C) of a [T][n] matrix into dst[C][ldd], zero past T. n a multiple of 8.
template <typename Tio>
__device__ void load_tile(float* dst, int ldd, const Tio* src, int t0, int T, int n) {
  const int n4 = n >> 2;
  for (int i = threadIdx.x; i < C * n4; i += kThreads) {
    const int r = i / n4, c = 4 * (i - r * n4);
    *reinterpret_cast<float4*>(dst + r * ldd + c) =
        t0 + r < T ? at4(src + (size_t)(t0 + r) * n + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

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
  __shared__ __align__(16) float A[C * LZ], Ab[C * LZ];
  const Dims& d = a.d;
  const int N = chunks(d.T), bh = blockIdx.x / N, n = blockIdx.x - bh * N;
  const int b = bh / d.H, h = bh - b * d.H;
  const size_t kh = (size_t)b * d.Hk + h / (d.H / d.Hk);
  const int ld = pad4(d.dk), t0 = n * C;
  float *K = sm, *Q = sm + C * ld;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) load_gates(g, a.beta, a.log_alpha, (size_t)bh * d.T, t0, d.T);
  load_tile(K, ld, static_cast<const Tio*>(a.k) + kh * d.T * d.dk, t0, d.T, d.dk);
  load_tile(Q, ld, static_cast<const Tio*>(a.q) + kh * d.T * d.dk, t0, d.T, d.dk);
  __syncthreads();
  const size_t cc = ((size_t)bh * N + n) * C * C;
  {  // a tile of 16 x 8 of K K^T and Q K^T per warp
    const int m0 = 16 * (warp & 1), n0 = 8 * (warp >> 1);
    float kk[4] = {0.f, 0.f, 0.f, 0.f}, qk[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < d.dk; c += 8) {
      const tf32::B8 kj = tf32::load_b<false>([&](int x, int j) { return K[(n0 + j) * ld + c + x]; });
      tf32::mma3<false>(kk, tf32::load_a([&](int i, int x) { return K[(m0 + i) * ld + c + x]; }), kj);
      tf32::mma3<false>(qk, tf32::load_a([&](int i, int x) { return Q[(m0 + i) * ld + c + x]; }), kj);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = m0 + (lane >> 2) + 8 * (e >> 1), j = n0 + 2 * (lane & 3) + (e & 1);
      const float m = j <= i ? decay(g, i, j) : 0.f, x = j < i ? m * kk[e] : 0.f;
      A[i * LZ + j] = x;
      Ab[i * LZ + j] = -x * g.beta[j];
      a.sv.P[cc + i * C + j] = a.scale * m * qk[e];
    }
  }
  if (warp == kWarps - 1) {
    WalkGates* wg = reinterpret_cast<WalkGates*>(a.sv.gates) + (size_t)bh * N + n;
    wg->beta[lane] = g.beta[lane];
    wg->G[lane] = g.G[lane];
    wg->w[lane] = g.w[lane];
    if (lane == 0) wg->GC = g.GC;
  }
  __syncthreads();
  // Z_ij = A_ij - sum_{j<m<i} A_im beta_m Z_mj: lane j owns column j (zero down to row j)
  if (warp == 0) {
    float z[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float s0 = A[i * LZ + lane], s1 = 0.f;
#pragma unroll
      for (int m = 0; m < i; m += 4) {
        const float4 b = at4(Ab + i * LZ + m);
        s0 = fmaf(b.x, z[m], s0);
        if (m + 1 < i) s1 = fmaf(b.y, z[m + 1], s1);
        if (m + 2 < i) s0 = fmaf(b.z, z[m + 2], s0);
        if (m + 3 < i) s1 = fmaf(b.w, z[m + 3], s1);
      }
      z[i] = s0 + s1;
      a.sv.Z[cc + i * C + lane] = z[i];
    }
  }
}

// ------------------------------------------------------------------ the walks
// One chunk's inputs in shared memory, two stages: the next chunk's copies (cp.async, in the
// I/O dtype) run while this one is worked on.
constexpr int LV = kRows + 8; // of V: 16-byte pieces in both types

template <typename Tio>
struct Stage {
  WalkGates* g;
  float *Z, *P;               // [C][LZ]
  Tio *K, *Q;                 // [C][padded dk]
  Tio* V;                     // [C][LV]: V or dY
};
// row stride of K and Q: whole 16-byte pieces, and an odd number of them
template <typename Tio>
__host__ __device__ constexpr int pad_row(int dk) { return dk + 16 / (int)sizeof(Tio); }
template <typename Tio>
__host__ __device__ constexpr size_t stage_bytes(int dk) {
  return sizeof(WalkGates) + 2 * C * LZ * sizeof(float) + (2 * C * pad_row<Tio>(dk) + C * LV) * sizeof(Tio);
}
template <typename Tio>
__device__ __forceinline__ Stage<Tio> stage_at(char* base, int s, int dk) {
  char* p = base + s * stage_bytes<Tio>(dk);
  Stage<Tio> g;
  g.g = reinterpret_cast<WalkGates*>(p);
  g.Z = reinterpret_cast<float*>(g.g + 1);
  g.P = g.Z + C * LZ;
  g.K = reinterpret_cast<Tio*>(g.P + C * LZ);
  g.Q = g.K + C * pad_row<Tio>(dk);
  g.V = g.Q + C * pad_row<Tio>(dk);
  return g;
}

__device__ __forceinline__ void copy16(void* dst, const void* src, bool ok) {
  const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
  const int n = ok ? 16 : 0;  // 0: filled with zeros
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// The pieces tid, tid + kThreads, .. of a matrix with `per` pieces in a row, without a division
// for each of them.
struct Pieces {
  int row, col, drow, dcol, per;
  __device__ Pieces(int per_row) : per(per_row) {
    row = threadIdx.x / per;
    col = threadIdx.x - row * per;
    drow = kThreads / per;
    dcol = kThreads - drow * per;
  }
  template <typename F>
  __device__ __forceinline__ void each(int rows, F f) const {
    for (int r = row, c = col; r < rows;) {
      f(r, c);
      r += drow;
      c += dcol;
      if (c >= per) c -= per, ++r;
    }
  }
};

// Asynchronous copies of chunk n (its 16-byte pieces over the CTA's threads).
template <typename Tio>
__device__ __forceinline__ void fetch(const Stage<Tio>& g, const Args& a, const Tio* v, size_t bh,
                                      size_t kh, int n, int n0, int rows, const Pieces& kp) {
  constexpr int E = 16 / sizeof(Tio);
  const Dims& d = a.d;
  const int N = chunks(d.T), t0 = n * C;
  const Tio* K = static_cast<const Tio*>(a.k) + kh * d.T * d.dk;
  const Tio* Q = static_cast<const Tio*>(a.q) + kh * d.T * d.dk;
  kp.each(C, [&](int t, int piece) {
    const int c = piece * E;
    const bool ok = t0 + t < d.T;
    const size_t at = (size_t)(ok ? t0 + t : 0) * d.dk + c;
    copy16(g.K + t * pad_row<Tio>(d.dk) + c, K + at, ok);
    copy16(g.Q + t * pad_row<Tio>(d.dk) + c, Q + at, ok);
  });
  constexpr int vc = kRows / E;
  for (int i = threadIdx.x; i < C * vc; i += kThreads) {
    const int t = i / vc, c = (i - t * vc) * E;
    const bool ok = t0 + t < d.T && c < rows;
    copy16(g.V + t * LV + c, ok ? v + (bh * d.T + t0 + t) * d.dv + n0 + c : v, ok);
  }
  const float* Z = a.sv.Z + (bh * N + n) * C * C;
  const float* P = a.sv.P + (bh * N + n) * C * C;
  const float* wg = a.sv.gates + (bh * N + n) * (sizeof(WalkGates) / sizeof(float));
  static_assert(sizeof(WalkGates) % 16 == 0 && sizeof(WalkGates) / 16 <= kThreads, "");
  if (threadIdx.x < sizeof(WalkGates) / 16)
    copy16(reinterpret_cast<float*>(g.g) + 4 * threadIdx.x, wg + 4 * threadIdx.x, true);
  static_assert(C * C / 4 == kThreads, "one piece of Z and P per thread");
  const int t = threadIdx.x / (C / 4), c = 4 * (threadIdx.x % (C / 4));
  copy16(g.Z + t * LZ + c, Z + t * C + c, true);
  copy16(g.P + t * LZ + c, P + t * C + c, true);
}

// Every product has the slice's 16 rows on one side, which is the height of a warp's tf32 tile
// (tf32.cuh). Warps 0 to 3 own 8 tokens each of S K^T, D and E, warps 4 to 7 the same tokens of
// S Q^T and y (backward: of dY P^T); for the update of S a warp owns every eighth 8 columns.
template <typename Tio, bool BWD>
__global__ void __launch_bounds__(kThreads) walk_kernel(Args a) {
  extern __shared__ __align__(16) char smc[];
  __shared__ float X[kRows * LZ], Y[kRows * LZ], U[kRows * LZ], W[kRows * LZ];  // [row][token]
  const Dims& d = a.d;
  const int N = chunks(d.T), ns = slices(d.dv), bh = blockIdx.x / ns;
  const int n0 = (blockIdx.x - bh * ns) * kRows;
  const int rows = min(kRows, d.dv - n0);
  const int b = bh / d.H, h = bh - b * d.H;
  const size_t kh = (size_t)b * d.Hk + h / (d.H / d.Hk);
  const int ld = pad4(d.dk), lk = pad_row<Tio>(d.dk);
  float* S = reinterpret_cast<float*>(smc + 2 * stage_bytes<Tio>(d.dk));  // [kRows][ld]
  const int tid = threadIdx.x, warp = tid >> 5;
  const int tr = (tid & 31) >> 2, tt = 8 * (warp & 3) + 2 * (tid & 3);  // this thread's part of a tile
  const bool second = warp >= 4;
  constexpr bool kExact = sizeof(Tio) == 2;
  const Tio* v = static_cast<const Tio*>(BWD ? a.dy : a.v);
  const bool fresh = a.log_alpha[(size_t)bh * d.T] < kResetLog;  // S0 may hold anything then
  for (int i = tid; i < kRows * d.dk; i += kThreads) {
    const int r = i / d.dk, c = i - r * d.dk;
    const size_t at = ((size_t)bh * d.dv + n0 + r) * d.dk + c;
    float s = 0.f;
    if (r < rows) {
      if (BWD)
        s = a.dST ? to_f32(static_cast<const Tio*>(a.dST)[at]) : 0.f;
      else
        s = a.S0 && !fresh ? a.S0[at] : 0.f;
    }
    S[r * ld + c] = s;
  }
  const Pieces kp(d.dk * (int)sizeof(Tio) / 16), sp(d.dk / 4);  // of rows of K and Q, of S
  auto at_chunk = [&](int c) { return BWD ? N - 1 - c : c; };
  fetch(stage_at<Tio>(smc, 0, d.dk), a, v, (size_t)bh, kh, at_chunk(0), n0, rows, kp);
  asm volatile("cp.async.commit_group;" ::: "memory");
  float* states = BWD ? a.dS : a.sv.S;
  for (int ci = 0; ci < N; ++ci) {
    const int n = at_chunk(ci), t0 = n * C;
    const Stage<Tio> st = stage_at<Tio>(smc, ci & 1, d.dk);
    const WalkGates& g = *st.g;
    if (ci + 1 < N)  // the other stage was last read before the barrier that ended chunk ci - 1
      fetch(stage_at<Tio>(smc, (ci + 1) & 1, d.dk), a, v, (size_t)bh, kh, at_chunk(ci + 1), n0, rows, kp);
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    if (states) {
      float* out = states + (((size_t)bh * N + n) * d.dv + n0) * d.dk;
      sp.each(rows, [&](int r, int c) {
        *reinterpret_cast<float4*>(out + r * d.dk + 4 * c) = at4(S + r * ld + 4 * c);
      });
    }
    const int n8 = 8 * (warp & 3);
    auto V = [&](int r, int t) { return to_f32(st.V[t * LV + r]); };
    auto store = [&](auto* out, const float (&x)[4]) {  // a tile of [row][token] to [t][d_v]
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = tr + 8 * (e >> 1), t = tt + (e & 1);
        if (t0 + t < d.T && r < rows) put(out + ((size_t)bh * d.T + t0 + t) * d.dv + n0 + r, x[e]);
      }
    };
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (!BWD || !second) {
      const Tio* B = !BWD && second ? st.Q : st.K;
      tf32::tile<kExact>(x, 0, d.dk, [&](int r, int k) { return S[r * ld + k]; },
                         [&](int k, int t) { return to_f32(B[(n8 + t) * lk + k]); });
    } else {  // P^T dY, and dY scaled for the update
      tf32::tile<false>(x, 0, C, [&](int r, int m) { return V(r, m); },
                        [&](int m, int t) { return st.P[m * LZ + n8 + t]; });
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = tr + 8 * (e >> 1), t = tt + (e & 1);
        Y[r * LZ + t] = x[e];
        W[r * LZ + t] = a.scale * g.G[t] * V(r, t);
      }
    }
    if (BWD) __syncthreads();
    if (!second) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = tr + 8 * (e >> 1), t = tt + (e & 1);
        // R = V - G S K; backward F = w dS K + P^T dY
        x[e] = BWD ? fmaf(g.w[t], x[e], Y[r * LZ + t]) : V(r, t) - g.G[t] * x[e];
        X[r * LZ + t] = -g.beta[t] * x[e];
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      // D = R - Z diag(beta) R; backward E = F - Z^T diag(beta) F
      tf32::tile<false>(x, 0, C, [&](int r, int m) { return X[r * LZ + m]; },
                        [&](int m, int t) { return BWD ? st.Z[m * LZ + n8 + t] : st.Z[(n8 + t) * LZ + m]; });
      float* wo = BWD ? a.E : a.sv.D;
      if (wo) store(wo, x);
      // U: what updates S (beta w D, -beta G E)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = tr + 8 * (e >> 1), t = tt + (e & 1);
        const float be = g.beta[t];
        U[r * LZ + t] = (BWD ? -be * g.G[t] : be * g.w[t]) * x[e];
        x[e] *= be;
        if (!BWD) Y[r * LZ + t] = x[e];
      }
      if (BWD) store(static_cast<Tio*>(a.dv_), x);
    }
    __syncthreads();
    if (!BWD && second) {  // y = scale G S Q^T + P diag(beta) D
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] *= a.scale * g.G[tt + (e & 1)];
      tf32::tile<false>(x, 0, C, [&](int r, int m) { return Y[r * LZ + m]; },
                        [&](int m, int t) { return st.P[(n8 + t) * LZ + m]; });
      if (a.y) store(static_cast<Tio*>(a.y), x);
    }
    // S <- G_C S + U K (+ scale G dY Q)
    const float GC = g.GC;
    for (int c0 = 8 * warp; c0 < d.dk; c0 += 8 * kWarps) {
      float* at = S + tr * ld + c0 + 2 * (tid & 3);
      float s[4] = {GC * at[0], GC * at[1], GC * at[8 * ld], GC * at[8 * ld + 1]};
      tf32::tile<kExact>(s, 0, C, [&](int r, int m) { return U[r * LZ + m]; },
                         [&](int m, int c) { return to_f32(st.K[m * lk + c0 + c]); });
      if (BWD)
        tf32::tile<kExact>(s, 0, C, [&](int r, int m) { return W[r * LZ + m]; },
                           [&](int m, int c) { return to_f32(st.Q[m * lk + c0 + c]); });
      at[0] = s[0];
      at[1] = s[1];
      at[8 * ld] = s[2];
      at[8 * ld + 1] = s[3];
    }
    __syncthreads();
  }
  if (BWD ? a.dS0 != nullptr : a.ST != nullptr)
    for (int i = tid; i < rows * d.dk; i += kThreads) {
      const size_t at = ((size_t)bh * d.dv + n0) * d.dk + i;
      const float s = S[(i / d.dk) * ld + i % d.dk];
      if (BWD)
        static_cast<Tio*>(a.dS0)[at] = from_f32<Tio>(s);
      else
        a.ST[at] = s;
    }
}

template <typename Tio>
size_t walk_smem(int dk) { return 2 * stage_bytes<Tio>(dk) + kRows * pad4(dk) * sizeof(float); }

// ------------------------------------------------------------------ gradients of q, k, gates
// One CTA per (chunk, key head). All products are warp tiles of 16 tokens and 8 columns (tf32.cuh):
// a warp has one of the tokens x tokens matrices and, of tokens x d_k, every fourth 8 columns, so
// sums over columns end in four lanes and four warps. The value heads that share the key head
// are walked in order and add up in registers.
constexpr int kVB = 16;       // rows of the states in shared memory at a time

template <typename Tio, int NJ>  // NJ: 32-column groups that cover dk
__global__ void __launch_bounds__(kThreads) grad_kernel(Args a) {
  extern __shared__ __align__(16) float sm[];
  __shared__ Gates g;
  __shared__ float X[C * LZ], Y[C * LZ], W[C * LD];  // W: X q.k - Y k.k
  __shared__ float dLx[4][C], dLz[4][C], red[kWarps];
  const Dims& d = a.d;
  const int N = chunks(d.T), n = blockIdx.x % N, t0 = n * C;
  const size_t kh = blockIdx.x / N;
  const int b = kh / d.Hk, hk = kh - (size_t)b * d.Hk, grp = d.H / d.Hk;
  const int ld = pad4(d.dk), lv = pad4(d.dv);
  float *K = sm, *Q = K + C * ld, *O = Q + C * ld, *D = O + C * lv, *E = D + C * lv;
  float *Sv = E + C * lv, *dSv = Sv + kVB * (d.dk + 8);
  const Pieces sp(d.dk / 4);  // of rows of S
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // this warp's tokens and columns, this thread's first of either
  const int m0 = 16 * (warp & 1), n0 = 8 * (warp >> 1);
  const int i0 = m0 + (lane >> 2), j0 = n0 + 2 * (lane & 3), lds = d.dk + 8;
  static_assert(2 * 16 == C && 8 * kWarps / 2 == C, "a tile of tokens x tokens per warp");
  load_tile(K, ld, static_cast<const Tio*>(a.k) + kh * d.T * d.dk, t0, d.T, d.dk);
  load_tile(Q, ld, static_cast<const Tio*>(a.q) + kh * d.T * d.dk, t0, d.T, d.dk);
  __syncthreads();
  float kk[4] = {0.f, 0.f, 0.f, 0.f}, qk[4] = {0.f, 0.f, 0.f, 0.f};  // k_i.k_j, q_i.k_j
  for (int c = 0; c < d.dk; c += 8) {
    const tf32::B8 kj = tf32::load_b<false>([&](int x, int j) { return K[(n0 + j) * ld + c + x]; });
    tf32::mma3<false>(kk, tf32::load_a([&](int i, int x) { return K[(m0 + i) * ld + c + x]; }), kj);
    tf32::mma3<false>(qk, tf32::load_a([&](int i, int x) { return Q[(m0 + i) * ld + c + x]; }), kj);
  }
  float aq[NJ][4], ak[NJ][4];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) aq[j][e] = ak[j][e] = 0.f;

  for (int hh = 0; hh < grp; ++hh) {
    const size_t bh = (size_t)b * d.H + hk * grp + hh;
    __syncthreads();
    if (warp == 0) load_gates(g, a.beta, a.log_alpha, bh * d.T, t0, d.T);
    load_tile(O, lv, static_cast<const Tio*>(a.dy) + bh * d.T * d.dv, t0, d.T, d.dv);
    load_tile(D, lv, a.sv.D + bh * d.T * d.dv, t0, d.T, d.dv);
    load_tile(E, lv, a.E + bh * d.T * d.dv, t0, d.T, d.dv);
    __syncthreads();
    const float* S = a.sv.S + (bh * N + n) * d.dv * d.dk;
    const float* dS = a.dS + (bh * N + n) * d.dv * d.dk;
    {  // X, Y, their part of dlog_alpha, dbeta
      float f[4] = {0.f, 0.f, 0.f, 0.f}, ed[4] = {0.f, 0.f, 0.f, 0.f};
      for (int c = 0; c < d.dv; c += 8) {
        const tf32::B8 dj = tf32::load_b<false>([&](int x, int j) { return D[(n0 + j) * lv + c + x]; });
        tf32::mma3<false>(f, tf32::load_a([&](int i, int x) { return O[(m0 + i) * lv + c + x]; }), dj);
        tf32::mma3<false>(ed, tf32::load_a([&](int i, int x) { return E[(m0 + i) * lv + c + x]; }), dj);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + 8 * (e >> 1), j = j0 + (e & 1);
        const float m = j <= i ? decay(g, i, j) * g.beta[j] : 0.f;
        const float x = a.scale * m * f[e], y = j < i ? m * g.beta[i] * ed[e] : 0.f;
        X[i * LZ + j] = x;
        Y[i * LZ + j] = y;
        W[i * LD + j] = j < i ? x * qk[e] - y * kk[e] : 0.f;
        if (i == j && t0 + i < d.T) static_cast<Tio*>(a.dbeta)[bh * d.T + t0 + i] = from_f32<Tio>(ed[e]);
      }
    }
    // dY S, E S, D dS
    float t[NJ][4], u[NJ][4], z[NJ][4];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) t[j][e] = u[j][e] = z[j][e] = 0.f;
    float ss = 0.f;
    for (int v0 = 0; v0 < d.dv; v0 += kVB) {  // kVB rows of S and dS at a time (dv may end inside)
      const int nv = min(kVB, d.dv - v0);
      __syncthreads();
      sp.each(nv, [&](int v, int c4) {
        const float4 s = at4(S + (size_t)(v0 + v) * d.dk + 4 * c4), ds = at4(dS + (size_t)(v0 + v) * d.dk + 4 * c4);
        *reinterpret_cast<float4*>(Sv + v * lds + 4 * c4) = s;
        *reinterpret_cast<float4*>(dSv + v * lds + 4 * c4) = ds;
        ss = dot4(s, ds, ss);
      });
      __syncthreads();
      for (int v = 0; v < nv; v += 8) {
        const tf32::A16 o = tf32::load_a([&](int i, int x) { return O[(m0 + i) * lv + v0 + v + x]; });
        const tf32::A16 ee = tf32::load_a([&](int i, int x) { return E[(m0 + i) * lv + v0 + v + x]; });
        const tf32::A16 dd = tf32::load_a([&](int i, int x) { return D[(m0 + i) * lv + v0 + v + x]; });
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int c0 = n0 + 32 * j;
          if (c0 >= d.dk) continue;
          const tf32::B8 s = tf32::load_b<false>([&](int x, int c) { return Sv[(v + x) * lds + c0 + c]; });
          const tf32::B8 ds = tf32::load_b<false>([&](int x, int c) { return dSv[(v + x) * lds + c0 + c]; });
          tf32::mma3<false>(t[j], o, s);
          tf32::mma3<false>(u[j], ee, s);
          tf32::mma3<false>(z[j], dd, ds);
        }
      }
    }
    ss = warp_sum(ss);
    if (lane == 0) red[warp] = ss;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // tokens i0 and i0 + 8
      const int i = i0 + 8 * h;
      const float cq = a.scale * g.G[i], ck = g.beta[i] * g.G[i], cz = g.beta[i] * g.w[i];
      float x = 0.f, zz = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        if (n0 + 32 * j >= d.dk) continue;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int e = 2 * h + y, c = j0 + 32 * j + y;
          const float qv = Q[i * ld + c], kv = K[i * ld + c];
          x += cq * t[j][e] * qv - ck * u[j][e] * kv;
          zz += cz * z[j][e] * kv;
          aq[j][e] += cq * t[j][e];
          ak[j][e] += cz * z[j][e] - ck * u[j][e];
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        zz += __shfl_xor_sync(0xffffffffu, zz, o);
      }
      if ((lane & 3) == 0) {
        dLx[warp >> 1][i] = x;
        dLz[warp >> 1][i] = zz;
      }
    }
    __syncthreads();
    for (int m = 0; m < C; m += 8) {  // dq += X K, dk += X^T Q - (Y + Y^T) K
      const tf32::A16 x = tf32::load_a([&](int i, int y) { return X[(m0 + i) * LZ + m + y]; });
      const tf32::A16 xt = tf32::load_a([&](int i, int y) { return X[(m + y) * LZ + m0 + i]; });
      const tf32::A16 yy = tf32::load_a([&](int i, int y) {
        return -(Y[(m0 + i) * LZ + m + y] + Y[(m + y) * LZ + m0 + i]);
      });
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int c0 = n0 + 32 * j;
        if (c0 >= d.dk) continue;
        const tf32::B8 kv = tf32::load_b<false>([&](int y, int c) { return K[(m + y) * ld + c0 + c]; });
        const tf32::B8 qv = tf32::load_b<false>([&](int y, int c) { return Q[(m + y) * ld + c0 + c]; });
        tf32::mma3<false>(aq[j], x, kv);
        tf32::mma3<false>(ak[j], xt, qv);
        tf32::mma3<false>(ak[j], yy, kv);
      }
    }
    if (warp == 0) {
      // token `lane`: the pairs (i >= t > j) by the running sum of column sums - row sums
      float rc = 0.f;
      for (int m = 0; m < C; ++m) rc += W[lane * LD + m] - W[m * LD + lane];
      float x = rc, zz = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        x += dLx[w][lane];
        zz += dLz[w][lane];
      }
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
    const int i = i0 + 8 * (e >> 1);
    const size_t row = (kh * d.T + t0 + i) * d.dk;
    if (t0 + i >= d.T) continue;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (n0 + 32 * j >= d.dk) continue;
      const int c = j0 + 32 * j + (e & 1);
      static_cast<Tio*>(a.dq)[row + c] = from_f32<Tio>(aq[j][e]);
      static_cast<Tio*>(a.dk_)[row + c] = from_f32<Tio>(ak[j][e]);
    }
  }
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// The shared memory of these kernels depends on d_k and d_v, so the opt-in is to all there is.
template <auto kKernel>
cudaError_t allow() {
  static std::atomic<uint64_t> done{0};
  return allow_smem(reinterpret_cast<const void*>(kKernel), done);
}

template <typename Tio, int NJ>
cudaError_t launch_grad(const Args& a, cudaStream_t st) {
  const size_t smem =
      ((size_t)C * (2 * pad4(a.d.dk) + 3 * pad4(a.d.dv)) + 2 * kVB * (a.d.dk + 8)) * sizeof(float);
  const cudaError_t e = allow<grad_kernel<Tio, NJ>>();
  if (e != cudaSuccess) return e;
  grad_kernel<Tio, NJ><<<chunks(a.d.T) * a.d.B * a.d.Hk, kThreads, smem, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename Tio>
cudaError_t fwd_t(const Args& a, cudaStream_t st) {
  const Dims& d = a.d;
  const size_t sp = (size_t)2 * C * pad4(d.dk) * sizeof(float);
  cudaError_t e = allow<prep_kernel<Tio>>();
  if (e != cudaSuccess) return e;
  prep_kernel<Tio><<<chunks(d.T) * d.B * d.H, kThreads, sp, st>>>(a);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const size_t sf = walk_smem<Tio>(d.dk);
  if ((e = allow<walk_kernel<Tio, false>>()) != cudaSuccess) return e;
  walk_kernel<Tio, false><<<slices(d.dv) * d.B * d.H, kThreads, sf, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename Tio>
cudaError_t bwd_t(const Args& a, cudaStream_t st) {
  const Dims& d = a.d;
  const size_t sf = walk_smem<Tio>(d.dk);
  cudaError_t e = allow<walk_kernel<Tio, true>>();
  if (e != cudaSuccess) return e;
  walk_kernel<Tio, true><<<slices(d.dv) * d.B * d.H, kThreads, sf, st>>>(a);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (d.dk <= 64) return launch_grad<Tio, 2>(a, st);
  if (d.dk <= 128) return launch_grad<Tio, 4>(a, st);
  return launch_grad<Tio, 8>(a, st);
}

}  // namespace

size_t saved_bytes(const Dims& d, bool states) {
  const size_t N = chunks(d.T), cc = up256(d.BH() * N * C * C * sizeof(float));
  size_t n = 2 * cc + up256(d.BH() * N * sizeof(WalkGates));
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
  s.gates = reinterpret_cast<float*>(base + 2 * cc);
  if (states) {
    base += 2 * cc + up256(d.BH() * N * sizeof(WalkGates));
    s.S = reinterpret_cast<float*>(base);
    s.D = reinterpret_cast<float*>(base + up256(d.BH() * N * d.dv * d.dk * sizeof(float)));
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
