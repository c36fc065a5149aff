// Norms of the queries and keys of each head, with the rotation by position in the same
// pass, and the gradients of both.
//
// Per (token, head) row x [d]:  r = 1 / sqrt(ss / n + eps) with ss = sum x^2 and n = 1 (L2)
// or d (RMS),  z = r x,  u = w z,  and for i < rot / 2 the pair (u_i, u_{i + rot/2}) is
// turned by the angle pos * inv_freq_i; columns from rot on stay.
// Backward, with g the turned-back gradient (the transpose of the turn):
//   dw = sum over rows of g z,   dx = r (g w - z (sum g w z) / n).
//
// Bound by memory: x (and dy) read once, y (dx) written once. A lane holds 8 consecutive
// columns (a 16-byte load of bf16), so a row of d columns takes the next power of two of
// d / 8 lanes, and rot a multiple of 16 puts a pair's partner into the same place of
// another lane of the row. The angles of a token are the same for all of its heads: a
// warp takes one token's rows in turn and computes them once. They are formed in double
// and reduced to a fraction of a turn there; a float32 product would be off by whole
// radians at far positions.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "gradlev.h"

namespace gradlev {
namespace qknorm {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int V = 8;           // columns per lane
constexpr int U = 4;           // rows of a lane group in flight
constexpr int kBwdCtas = 148 * 4;  // fixed: the weights' gradients add up in a fixed order

struct Rows {                  // queries or keys
  const void* x;               // [B,T,H,d] by strides (elements)
  long long sb, st, sh;
  const float* w;              // [d] or null (1)
  void* y;                     // forward output [B,H,T,d]
  const void* dy;              // backward input [B,H,T,d]
  void* dx;                    // backward output, by strides
  long long db, dt, dh;
  int H;
};

struct NormArgs {
  int B, T, d, half, items;    // items: pieces that a token's rows are cut into (forward)
  float inv_n, eps;
  Rows r[2];
  const int* pos;              // [B,T] or null (t)
  const float* inv_freq;       // [half]
  float* part;                 // [kBwdCtas][2][d]: the weights' gradients, or null
};

struct F8 { float v[V]; };

__device__ __forceinline__ F8 load8(const __nv_bfloat16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t a[4] = {u.x, u.y, u.z, u.w};
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.v[2 * i] = __uint_as_float(a[i] << 16);
    f.v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
  return f;
}
__device__ __forceinline__ F8 load8(const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const F8& f) {
  uint32_t a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.v[2 * i], f.v[2 * i + 1]);
    a[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(a[0], a[1], a[2], a[3]);
}
__device__ __forceinline__ void store8(float* p, const F8& f) {
  *reinterpret_cast<float4*>(p) = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f.v[4], f.v[5], f.v[6], f.v[7]);
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The turn of this lane's 8 columns: out = c u + s u_partner (forward sign of s; the
// transpose uses -s). c = 1 and s = 0 outside the rotated columns.
struct Turn {
  float c[V], s[V];
  int partner;   // lane within the group
};

__device__ __forceinline__ Turn make_turn(const NormArgs& a, int gl, size_t bt, int t) {
  Turn u;
  const int c0 = V * gl;
  u.partner = gl;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    u.c[i] = 1.f;
    u.s[i] = 0.f;
  }
  if (c0 < 2 * a.half) {
    const bool lo = c0 < a.half;
    const int i0 = lo ? c0 : c0 - a.half;
    u.partner = lo ? gl + a.half / V : gl - a.half / V;
    const double pos = a.pos ? (double)a.pos[bt] : (double)t;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      double turns = pos * (double)a.inv_freq[i0 + i] * 0.15915494309189533577;  // / 2 pi
      turns -= rint(turns);
      float s, c;
      sincospif((float)(2.0 * turns), &s, &c);
      u.c[i] = c;
      u.s[i] = lo ? -s : s;
    }
  }
  return u;
}

template <int G>
__device__ __forceinline__ F8 apply_turn(const Turn& u, const F8& x, int gbase, float sign) {
  F8 y;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float p = __shfl_sync(0xffffffffu, x.v[i], gbase + u.partner);
    y.v[i] = fmaf(u.c[i], x.v[i], sign * u.s[i] * p);
  }
  return y;
}

__device__ __forceinline__ F8 weights(const float* w, int c0, int d) {
  F8 f;
#pragma unroll
  for (int i = 0; i < V; ++i) f.v[i] = w && c0 < d ? w[c0 + i] : 1.f;
  return f;
}

// ------------------------------------------------------------------ forward
// A warp takes `items`-th parts of a token's rows (queries, then keys).
template <typename Tio, int G>
__global__ void __launch_bounds__(kThreads) fwd_kernel(NormArgs a) {
  constexpr int R = 32 / G;  // rows a warp takes at a time
  const int lane = threadIdx.x & 31, gl = lane % G, gbase = lane - gl, c0 = V * gl;
  const size_t id = (size_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const size_t bt = id / a.items;
  if (bt >= (size_t)a.B * a.T) return;
  const int item = id - bt * a.items;
  const int b = bt / a.T, t = bt - (size_t)b * a.T;
  const int rows = a.r[0].H + a.r[1].H;
  const int per = (rows + a.items - 1) / a.items;
  const int lo = item * per, hi = min(rows, lo + per);
  const Turn turn = make_turn(a, gl, bt, t);
  const F8 w0 = weights(a.r[0].w, c0, a.d), w1 = weights(a.r[1].w, c0, a.d);
  const bool in = c0 < a.d;
  for (int base = lo; base < hi; base += R * U) {
    F8 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = base + u * R + lane / G;
      const int which = row >= a.r[0].H;
      const Rows& r = a.r[which];
      const int h = row - (which ? a.r[0].H : 0);
      if (in && row < hi)
        x[u] = load8(static_cast<const Tio*>(r.x) + b * r.sb + t * r.st + h * r.sh + c0);
      else
        x[u] = F8{};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = base + u * R + lane / G;
      const int which = row >= a.r[0].H;
      const int h = row - (which ? a.r[0].H : 0);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) ss = fmaf(x[u].v[i], x[u].v[i], ss);
      const float rs = 1.f / sqrtf(fmaf(group_sum<G>(ss), a.inv_n, a.eps));
#pragma unroll
      for (int i = 0; i < V; ++i) x[u].v[i] *= rs * (which ? w1.v[i] : w0.v[i]);
      const F8 y = apply_turn<G>(turn, x[u], gbase, 1.f);
      if (in && row < hi)
        store8(static_cast<Tio*>(a.r[which].y) + (((size_t)b * a.r[which].H + h) * a.T + t) * a.d + c0, y);
    }
  }
}

// ------------------------------------------------------------------ backward
// kBwdCtas CTAs walk the tokens with a fixed stride; each lane adds up the weights'
// gradients of its columns and each CTA leaves one partial per weight.
template <typename Tio, int G>
__global__ void __launch_bounds__(kThreads) bwd_kernel(NormArgs a) {
  constexpr int R = 32 / G;
  __shared__ float acc[2][kWarps][32 / G][G * V];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane % G, gbase = lane - gl, c0 = V * gl;
  const bool in = c0 < a.d;
  const int rows = a.r[0].H + a.r[1].H;
  F8 dw0{}, dw1{};
  const size_t tokens = (size_t)a.B * a.T;
  for (size_t bt = (size_t)blockIdx.x * kWarps + warp; bt < tokens; bt += (size_t)gridDim.x * kWarps) {
    const int b = bt / a.T, t = bt - (size_t)b * a.T;
    const Turn turn = make_turn(a, gl, bt, t);
    for (int base = 0; base < rows; base += R) {
      const int row = base + lane / G;
      const int which = row >= a.r[0].H;
      const Rows& r = a.r[which];
      const int h = row - (which ? a.r[0].H : 0);
      const bool ok = in && row < rows;
      F8 x{}, g{};
      if (ok) {
        x = load8(static_cast<const Tio*>(r.x) + b * r.sb + t * r.st + h * r.sh + c0);
        g = load8(static_cast<const Tio*>(r.dy) + (((size_t)b * r.H + h) * a.T + t) * a.d + c0);
      }
      g = apply_turn<G>(turn, g, gbase, -1.f);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) ss = fmaf(x.v[i], x.v[i], ss);
      const float rs = 1.f / sqrtf(fmaf(group_sum<G>(ss), a.inv_n, a.eps));
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x.v[i] *= rs;  // z
        const float gz = g.v[i] * x.v[i];
        if (row < rows) {
          dw0.v[i] += which ? 0.f : gz;
          dw1.v[i] += which ? gz : 0.f;
        }
        if (r.w && ok) g.v[i] *= r.w[c0 + i];
        dot = fmaf(g.v[i], x.v[i], dot);
      }
      dot = group_sum<G>(dot) * a.inv_n;
#pragma unroll
      for (int i = 0; i < V; ++i) g.v[i] = rs * fmaf(-dot, x.v[i], g.v[i]);
      if (ok) store8(static_cast<Tio*>(r.dx) + b * r.db + t * r.dt + h * r.dh + c0, g);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    acc[0][warp][lane / G][c0 + i] = dw0.v[i];
    acc[1][warp][lane / G][c0 + i] = dw1.v[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.d; i += kThreads) {
    const int which = i / a.d, c = i - which * a.d;
    float s = 0.f;
    for (int w = 0; w < kWarps; ++w)
      for (int g = 0; g < 32 / G; ++g) s += acc[which][w][g][c];
    a.part[(size_t)blockIdx.x * 2 * a.d + i] = s;
  }
}

// One warp per column: the partials in a fixed order.
__global__ void __launch_bounds__(kThreads) reduce_kernel(const float* part, int ctas, int d,
                                                          float* dwq, float* dwk) {
  const int col = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (col >= 2 * d) return;
  float* out = col < d ? dwq : dwk;
  if (!out) return;
  double s = 0.0;
  for (int i = lane; i < ctas; i += 32) s += (double)part[(size_t)i * 2 * d + col];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) out[col < d ? col : col - d] = (float)s;
}

template <typename Tio, int G>
cudaError_t launch(NormArgs a, bool bwd, cudaStream_t st) {
  const size_t tokens = (size_t)a.B * a.T;
  if (!bwd) {
    // few tokens: a token's rows are cut into up to one group of rows per warp
    const int rows = a.r[0].H + a.r[1].H, most = (rows + 32 / G - 1) / (32 / G);
    a.items = 1;
    while (a.items < most && tokens * a.items < 148 * 4 * 8) a.items *= 2;
    const size_t warps = tokens * a.items;
    fwd_kernel<Tio, G><<<(unsigned)((warps + kWarps - 1) / kWarps), kThreads, 0, st>>>(a);
  } else {
    bwd_kernel<Tio, G><<<kBwdCtas, kThreads, 0, st>>>(a);
  }
  count_launch();
  return cudaGetLastError();
}

template <typename Tio>
cudaError_t launch_t(const NormArgs& a, bool bwd, cudaStream_t st) {
  const int lanes = a.d / V;
  if (lanes <= 4) return launch<Tio, 4>(a, bwd, st);
  if (lanes <= 8) return launch<Tio, 8>(a, bwd, st);
  if (lanes <= 16) return launch<Tio, 16>(a, bwd, st);
  return launch<Tio, 32>(a, bwd, st);
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

gradlev_status check(int B, int T, int Hq, int Hk, int d, int rot, gradlev_dtype dt, int norm) {
  if (B <= 0 || T <= 0 || Hq <= 0 || Hk <= 0 || d <= 0 || rot < 0) return GRADLEV_ERR_INVALID_ARG;
  if (dt != GRADLEV_F32 && dt != GRADLEV_BF16) return GRADLEV_ERR_INVALID_ARG;
  if (norm != GRADLEV_NORM_L2 && norm != GRADLEV_NORM_RMS) return GRADLEV_ERR_INVALID_ARG;
  if (d % V != 0 || d > 32 * V || rot % (2 * V) != 0 || rot > d) return GRADLEV_ERR_UNSUPPORTED;
  if ((long long)B * T * ((long long)Hq + Hk) >= (1LL << 31)) return GRADLEV_ERR_UNSUPPORTED;
  return GRADLEV_OK;
}

// Strides of 16-byte-loadable rows.
bool strides_ok(const long long* s, size_t es) {
  if (!s) return false;
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || (s[i] * (long long)es) % 16 != 0) return false;
  return true;
}

Rows rows_of(const void* x, const long long* s, const float* w, int H) {
  Rows r{};
  r.x = x;
  r.sb = s[0];
  r.st = s[1];
  r.sh = s[2];
  r.w = w;
  r.H = H;
  return r;
}

}  // namespace
}  // namespace qknorm
}  // namespace gradlev

using namespace gradlev;
using namespace gradlev::qknorm;

extern "C" {

size_t gradlev_qk_norm_rope_workspace_bytes(int B, int T, int Hq, int Hk, int d, gradlev_dtype dt) {
  if (check(B, T, Hq, Hk, d, 0, dt, GRADLEV_NORM_L2) != GRADLEV_OK) return 0;
  return 256 + (size_t)kBwdCtas * 2 * d * sizeof(float);
}

gradlev_status gradlev_qk_norm_rope_fwd(int B, int T, int Hq, int Hk, int d, int rot,
                                        gradlev_dtype dt, int norm, float eps, const void* q,
                                        const long long* q_strides, const void* k,
                                        const long long* k_strides, const float* wq,
                                        const float* wk, const int* pos, const float* inv_freq,
                                        void* yq, void* yk, void* stream) {
  reset_launch_count();
  const gradlev_status s = check(B, T, Hq, Hk, d, rot, dt, norm);
  if (s != GRADLEV_OK) return s;
  const size_t es = dt == GRADLEV_BF16 ? 2 : 4;
  if (!q || !k || !yq || !yk || (rot > 0 && !inv_freq) || !(eps >= 0.f)) return GRADLEV_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(yq, 16) || !aligned(yk, 16) ||
      !aligned(wq, 4) || !aligned(wk, 4) || !aligned(pos, 4) || !aligned(inv_freq, 4) ||
      !strides_ok(q_strides, es) || !strides_ok(k_strides, es))
    return GRADLEV_ERR_INVALID_ARG;
  NormArgs a{B, T, d, rot / 2, 1, norm == GRADLEV_NORM_RMS ? 1.f / d : 1.f, eps};
  a.r[0] = rows_of(q, q_strides, wq, Hq);
  a.r[1] = rows_of(k, k_strides, wk, Hk);
  a.r[0].y = yq;
  a.r[1].y = yk;
  a.pos = pos;
  a.inv_freq = inv_freq;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dt == GRADLEV_BF16 ? launch_t<__nv_bfloat16>(a, false, st)
                                           : launch_t<float>(a, false, st);
  return e == cudaSuccess ? GRADLEV_OK : GRADLEV_ERR_CUDA;
}

gradlev_status gradlev_qk_norm_rope_bwd(
    int B, int T, int Hq, int Hk, int d, int rot, gradlev_dtype dt, int norm, float eps,
    const void* dyq, const void* dyk, const void* q, const long long* q_strides, const void* k,
    const long long* k_strides, const float* wq, const float* wk, const int* pos,
    const float* inv_freq, void* dq, const long long* dq_strides, void* dk,
    const long long* dk_strides, float* dwq, float* dwk, void* workspace, size_t ws_bytes,
    void* stream) {
  reset_launch_count();
  const gradlev_status s = check(B, T, Hq, Hk, d, rot, dt, norm);
  if (s != GRADLEV_OK) return s;
  const size_t es = dt == GRADLEV_BF16 ? 2 : 4;
  if (!dyq || !dyk || !q || !k || !dq || !dk || (rot > 0 && !inv_freq) || !(eps >= 0.f) ||
      (wq == nullptr) != (dwq == nullptr) || (wk == nullptr) != (dwk == nullptr))
    return GRADLEV_ERR_INVALID_ARG;
  for (const void* p : {dyq, dyk, q, k, (const void*)dq, (const void*)dk})
    if (!aligned(p, 16)) return GRADLEV_ERR_INVALID_ARG;
  for (const void* p : {(const void*)wq, (const void*)wk, (const void*)dwq, (const void*)dwk,
                        (const void*)pos, (const void*)inv_freq})
    if (!aligned(p, 4)) return GRADLEV_ERR_INVALID_ARG;
  for (const long long* t : {q_strides, k_strides, dq_strides, dk_strides})
    if (!strides_ok(t, es)) return GRADLEV_ERR_INVALID_ARG;
  const bool dw = dwq || dwk;
  if (dw && (!workspace || !aligned(workspace, 256))) return GRADLEV_ERR_INVALID_ARG;
  if (dw && ws_bytes < gradlev_qk_norm_rope_workspace_bytes(B, T, Hq, Hk, d, dt))
    return GRADLEV_ERR_WORKSPACE;
  NormArgs a{B, T, d, rot / 2, 1, norm == GRADLEV_NORM_RMS ? 1.f / d : 1.f, eps};
  a.r[0] = rows_of(q, q_strides, wq, Hq);
  a.r[1] = rows_of(k, k_strides, wk, Hk);
  a.r[0].dy = dyq;
  a.r[1].dy = dyk;
  a.r[0].dx = dq;
  a.r[1].dx = dk;
  for (int i = 0; i < 2; ++i) {
    const long long* t = i ? dk_strides : dq_strides;
    a.r[i].db = t[0];
    a.r[i].dt = t[1];
    a.r[i].dh = t[2];
  }
  a.pos = pos;
  a.inv_freq = inv_freq;
  a.part = dw ? reinterpret_cast<float*>(static_cast<char*>(workspace) + 256) : nullptr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = dt == GRADLEV_BF16 ? launch_t<__nv_bfloat16>(a, true, st)
                                     : launch_t<float>(a, true, st);
  if (e == cudaSuccess && dw) {
    reduce_kernel<<<(2 * d + kWarps - 1) / kWarps, kThreads, 0, st>>>(a.part, kBwdCtas, d, dwq, dwk);
    count_launch();
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? GRADLEV_OK : GRADLEV_ERR_CUDA;
}

}  // extern "C"
