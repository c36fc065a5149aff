// Norms of the queries and keys of each head, with the rotation by position in the same
// pass, and the gradients of both.
//
// Per (token, head) row x [d]:  r = 1 / sqrt(ss / n + eps) with ss = sum x^2 and n = 1 (L2)
// or d (RMS),  z = r x,  u = w z,  and for i < rot / 2 the pair (u_i, u_{i + rot/2}) is
// turned by the angle pos * inv_freq_i; columns from rot on stay.
// Backward, with g the turned-back gradient (the transpose of the turn):
//   dw = sum over rows of g z,   dx = r (g w - z (sum g w z) / n).
//
// Bound by memory: x (and dy) read once, y (dx) written once. A lane holds 8 columns of a
// row, 4 in each of two places that the rotation pairs up (i and i + rot / 2; past the
// rotated columns simply 8 in a row), so that the turn needs no exchange between lanes and
// a lane only forms 4 angles. A row takes the next power of two of d / 8 lanes. The angles
// of a token are the same for all of its heads: a warp takes one token's rows in turn and
// computes them once.
//
// Angles: pos * inv_freq is off by whole radians in float32 at far positions. Only the
// fraction of a turn matters, so inv_freq / 2 pi goes into a 64-bit binary fraction F once
// per lane, and pos * F modulo 2^64 is that fraction, exact up to F's own rounding.
//
// Measured with 16 + 16 heads of 128, bf16: forward 110 us for B8 T4096 (537 MB, 4.9 TB/s),
// backward 173 + 7 us (806 MB, 4.6 TB/s).
// What the bandwidth needs is loads in flight: 8 rows of bf16 per lane group (kept as
// loaded) at 16 warps per SM move 537 MB (B8 T4096, 16 + 16 heads of 128) in 110 us;
// 4 rows at 24 warps took 128 us, and 4 unpacked rows at 20 warps 218 us.
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
constexpr int kFwdCtas = 148 * 8, kBwdCtas = 148 * 4;  // the latter fixed: the weights'
                               // gradients add up in a fixed order

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

struct F8 { float v[V]; };   // columns [ca, ca + 4), [cb, cb + 4)

// A lane's columns of a row as loaded: rows in flight cost half the registers that way. Plain
// loads: the gradients may be written over the rows they are formed from.
template <typename Tio> struct Raw;
template <> struct Raw<__nv_bfloat16> {
  uint2 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* pa, const __nv_bfloat16* pb) {
    a = *reinterpret_cast<const uint2*>(pa);
    b = *reinterpret_cast<const uint2*>(pb);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint2(0u, 0u); }
  __device__ __forceinline__ F8 get() const {
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
    F8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.v[2 * i] = __uint_as_float(w[i] << 16);
      f.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return f;
  }
};
template <> struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* pa, const float* pb) {
    a = *reinterpret_cast<const float4*>(pa);
    b = *reinterpret_cast<const float4*>(pb);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ F8 get() const { return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
};
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Where this lane's columns are, and the binary fractions of its 4 angles (zero outside the
// rotated columns, which leaves them as they are).
struct Lane {
  int ca, cb;
  bool in, turns;
  unsigned long long F[4];
};

__device__ __forceinline__ Lane make_lane(const NormArgs& a, int gl) {
  Lane l;
  l.in = V * gl < a.d;
  l.turns = 4 * gl < a.half;
  l.ca = l.turns ? 4 * gl : V * gl;
  l.cb = l.turns ? a.half + 4 * gl : V * gl + 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    l.F[i] = 0;
    if (l.turns) {
      double f = (double)a.inv_freq[l.ca + i] * 0.15915494309189533577;  // / 2 pi
      f -= floor(f);
      l.F[i] = f < 1.0 ? (unsigned long long)(f * 18446744073709551616.0) : 0ull;
    }
  }
  return l;
}

struct Turn { float c[4], s[4]; };

__device__ __forceinline__ Turn make_turn(const NormArgs& a, const Lane& l, size_t bt, int t) {
  Turn u;
  const long long pos = a.pos ? a.pos[bt] : t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the top 32 bits, signed: half turns times 2^31
    const int hi = (int)(((unsigned long long)pos * l.F[i]) >> 32);
    u.c[i] = 1.f;
    u.s[i] = 0.f;
    if (l.turns) sincospif((float)hi * 0x1p-31f, &u.s[i], &u.c[i]);
  }
  return u;
}

__device__ __forceinline__ F8 weights(const float* w, const Lane& l) {
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.v[i] = w && l.in ? w[l.ca + i] : 1.f;
    f.v[4 + i] = w && l.in ? w[l.cb + i] : 1.f;
  }
  return f;
}

template <typename Tio>
__device__ __forceinline__ Raw<Tio> load_row(const Tio* p, const Lane& l, bool ok) {
  Raw<Tio> x;
  x.zero();
  if (ok) x.load(p + l.ca, p + l.cb);
  return x;
}
template <typename Tio>
__device__ __forceinline__ void store_row(Tio* p, const Lane& l, const F8& x) {
  store4(p + l.ca, x.v);
  store4(p + l.cb, x.v + 4);
}

// ------------------------------------------------------------------ forward
// A warp takes `items`-th parts of a token's rows (queries, then keys), U rows of each lane
// group in flight. The weights ride on the turn: 16 products per token and list instead of
// 8 per row.
template <typename Tio, int G>
__global__ void __launch_bounds__(kThreads, 4) fwd_kernel(NormArgs a) {
  // rows a warp takes at a time, and how many of those are in flight
  constexpr int R = 32 / G, U = sizeof(Tio) == 2 ? 8 : 4;
  const int lane = threadIdx.x & 31;
  const Lane l = make_lane(a, lane % G);
  const int rows = a.r[0].H + a.r[1].H;
  const int per = (rows + a.items - 1) / a.items;
  const size_t work = (size_t)a.B * a.T * a.items;
  for (size_t id = (size_t)blockIdx.x * kWarps + (threadIdx.x >> 5); id < work;
       id += (size_t)gridDim.x * kWarps) {
    const size_t bt = id / a.items;
    const int item = id - bt * a.items;
    const int b = bt / a.T, t = bt - (size_t)b * a.T;
    const Turn turn = make_turn(a, l, bt, t);
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const Rows& r = a.r[which];
      const int first = which ? a.r[0].H : 0;
      const int lo = max(item * per - first, 0), hi = min((item + 1) * per - first, r.H);
      if (lo >= hi) continue;
      const F8 w = weights(r.w, l);
      const Tio* x0 = static_cast<const Tio*>(r.x) + b * r.sb + t * r.st;
      Tio* y0 = static_cast<Tio*>(r.y) + ((size_t)b * r.H * a.T + t) * a.d;
      const size_t yh = (size_t)a.T * a.d;
      for (int base = lo; base < hi; base += R * U) {
        Raw<Tio> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = base + u * R + lane / G;
          raw[u] = load_row(x0 + h * r.sh, l, l.in && h < hi);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = base + u * R + lane / G;
          const F8 x = raw[u].get();
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < V; ++i) ss = fmaf(x.v[i], x.v[i], ss);
          const float rs = rsqrtf(fmaf(group_sum<G>(ss), a.inv_n, a.eps));
          F8 y;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = x.v[i] * rs, q = x.v[4 + i] * rs;
            y.v[i] = fmaf(turn.c[i] * w.v[i], p, -(turn.s[i] * w.v[4 + i]) * q);
            y.v[4 + i] = fmaf(turn.c[i] * w.v[4 + i], q, turn.s[i] * w.v[i] * p);
          }
          if (l.in && h < hi) store_row(y0 + h * yh, l, y);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ backward
// kBwdCtas CTAs walk the tokens with a fixed stride; each lane adds up the weights'
// gradients of its columns and each CTA leaves one partial per weight. Both sums of a row
// are taken over x as it is, in one round of exchanges:
//   sum g w z = r sum g w x.
template <typename Tio, int G>
__global__ void __launch_bounds__(kThreads, 4) bwd_kernel(NormArgs a) {
  constexpr int R = 32 / G, U = sizeof(Tio) == 2 ? 4 : 2;
  __shared__ float acc[2][kWarps][R][G * V];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Lane l = make_lane(a, lane % G);
  const size_t tokens = (size_t)a.B * a.T;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const Rows& r = a.r[which];
    const F8 w = weights(r.w, l);
    F8 dw{};
    for (size_t bt = (size_t)blockIdx.x * kWarps + warp; bt < tokens;
         bt += (size_t)gridDim.x * kWarps) {
      const int b = bt / a.T, t = bt - (size_t)b * a.T;
      const Turn turn = make_turn(a, l, bt, t);
      const Tio* x0 = static_cast<const Tio*>(r.x) + b * r.sb + t * r.st;
      const Tio* g0 = static_cast<const Tio*>(r.dy) + ((size_t)b * r.H * a.T + t) * a.d;
      Tio* d0 = static_cast<Tio*>(r.dx) + b * r.db + t * r.dt;
      const size_t gh = (size_t)a.T * a.d;
      for (int base = 0; base < r.H; base += R * U) {
        Raw<Tio> xs[U], gs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = base + u * R + lane / G;
          const bool ok = l.in && h < r.H;
          xs[u] = load_row(x0 + h * r.sh, l, ok);
          gs[u] = load_row(g0 + h * gh, l, ok);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = base + u * R + lane / G;
          const F8 x = xs[u].get(), gy = gs[u].get();
          F8 g;
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // turned back
            g.v[i] = fmaf(turn.c[i], gy.v[i], turn.s[i] * gy.v[4 + i]);
            g.v[4 + i] = fmaf(turn.c[i], gy.v[4 + i], -turn.s[i] * gy.v[i]);
          }
          float ss = 0.f, gx = 0.f;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            ss = fmaf(x.v[i], x.v[i], ss);
            gx = fmaf(g.v[i] * w.v[i], x.v[i], gx);
          }
#pragma unroll
          for (int o = G / 2; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            gx += __shfl_xor_sync(0xffffffffu, gx, o);
          }
          const float rs = rsqrtf(fmaf(ss, a.inv_n, a.eps));
          const bool ok = l.in && h < r.H;
          const float m = -gx * rs * rs * a.inv_n;  // dx = r (g w + m x)
          const float rz = ok ? rs : 0.f;           // a row past the end may have r = inf
          F8 y;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            dw.v[i] = fmaf(g.v[i] * rz, x.v[i], dw.v[i]);
            y.v[i] = rs * fmaf(m, x.v[i], g.v[i] * w.v[i]);
          }
          if (ok) store_row(d0 + h * r.dh, l, y);
        }
      }
    }
    if (a.part && l.in) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[which][warp][lane / G][l.ca + i] = dw.v[i];
        acc[which][warp][lane / G][l.cb + i] = dw.v[4 + i];
      }
    }
  }
  if (!a.part) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.d; i += kThreads) {
    const int which = i / a.d, c = i - which * a.d;
    float s = 0.f;
    for (int w = 0; w < kWarps; ++w)
      for (int g = 0; g < R; ++g) s += acc[which][w][g][c];
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
    const size_t ctas = (tokens * a.items + kWarps - 1) / kWarps;
    fwd_kernel<Tio, G><<<(unsigned)(ctas < kFwdCtas ? ctas : kFwdCtas), kThreads, 0, st>>>(a);
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
  const long long BT = (long long)B * T, heads = (long long)Hq + Hk;
  if (BT >= 1LL << 31 || BT * heads >= 1LL << 31) return GRADLEV_ERR_UNSUPPORTED;
  return GRADLEV_OK;
}

// Strides of 16-byte-loadable rows.
bool strides_ok(const long long* s, size_t es) {
  if (!s) return false;
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || (s[i] * (long long)es) % 16 != 0) return false;
  return true;
}

// Rows that are written: none of them twice by a stride of zero.
bool rows_apart(const long long* s, int B, int T, int H) {
  return (s[0] != 0 || B == 1) && (s[1] != 0 || T == 1) && (s[2] != 0 || H == 1);
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
  if (!rows_apart(dq_strides, B, T, Hq) || !rows_apart(dk_strides, B, T, Hk))
    return GRADLEV_ERR_INVALID_ARG;
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
