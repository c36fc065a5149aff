// The gated delta rule token by token, on states that stay in device memory (serving).
// Formulas in delta.h. The rows of S are independent given q_t and k_t, so a lane group
// owns kRows rows and keeps them in float32 registers across the T tokens of the call.
// y needs no second pass over the updated row:
//   S' = a S,  e = v - S' k,  y = scale (S' q + beta e (k.q)),  S <- S' + beta e k^T,
// so a token costs one round of sums over the lanes (S'k, S'q and k.q together).
//
// Bound by memory: S is read once and written once per call, everything else is small: 118 MB
// for 56 requests (and 8 padding rows) of 16 heads of 128 x 128, 24.2 us or 4.9 TB/s (30 us with
// a butterfly for every row, which costs 80 exchanges where the halves take 25). A single
// request's 16 heads take 3.2 us, the latency of loads, sums and stores.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "delta.h"
#include "gradlev.h"

namespace gradlev {
namespace delta {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxDk = 256;

struct StepArgs {
  int B, H, Hk, T, dk, dv, P;
  const void *q, *k, *v;          // [B,Hk,T,dk], [B,Hk,T,dk], [B,H,T,dv]
  const float *beta, *log_alpha;  // [B,H,T]
  float scale;
  const int* slots;               // [B] rows of the pool, or null (row b)
  float* S;                       // [P,H,dv,dk]
  void* y;                        // [B,H,T,dv]
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

// Sum over the LPR lanes of a group; every lane ends with the same value.
template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// LPR lanes share a row, NK4 float4 of it per lane (dk <= 4 LPR NK4); kRows rows per lane group.
template <typename Tio, int LPR, int NK4, int kRows>
__global__ void __launch_bounds__(kWarps * 32) step_kernel(StepArgs a) {
  constexpr int kGroups = 32 / LPR, kRowsPerCta = kWarps * kGroups * kRows;
  const int lane = threadIdx.x & 31, gl = lane % LPR;
  const int tiles = (a.dv + kRowsPerCta - 1) / kRowsPerCta;
  const int bh = blockIdx.x / tiles, tile = blockIdx.x - bh * tiles;
  const int b = bh / a.H, h = bh - b * a.H;
  const int nb = tile * kRowsPerCta + (threadIdx.x / LPR) * kRows;  // first row of this group
  const int dk = a.dk;
  bool kok[NK4];
#pragma unroll
  for (int i = 0; i < NK4; ++i) kok[i] = 4 * (gl + LPR * i) < dk;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const size_t kt = ((size_t)b * a.Hk + h / (a.H / a.Hk)) * a.T;
  const Tio* qg = static_cast<const Tio*>(a.q) + kt * dk;
  const Tio* kg = static_cast<const Tio*>(a.k) + kt * dk;
  const Tio* vg = static_cast<const Tio*>(a.v) + (size_t)bh * a.T * a.dv;
  // The sums over a group's lanes go by halves: an exchange leaves each lane with half of the values
  // (those of S'k in the lower lanes, of S'q in the upper ones), until each has one row's.
  constexpr int kHalf = LPR / 2, kSpread = kHalf / kRows;  // lanes per row in either half
  static_assert(kSpread >= 1 && kSpread * kRows == kHalf, "a lane ends with one value");
  const int own = nb + (gl & (kHalf - 1)) / kSpread;
  // a token's vectors, loaded one token ahead (the first while the slot is looked up)
  float4 qn[NK4], kn[NK4];
  float vn, bn, ln;  // v of this lane's own row (below)
  auto load_token = [&](int t) {
#pragma unroll
    for (int i = 0; i < NK4; ++i) {
      qn[i] = kok[i] ? load4(qg + (size_t)t * dk + 4 * (gl + LPR * i)) : zero;
      kn[i] = kok[i] ? load4(kg + (size_t)t * dk + 4 * (gl + LPR * i)) : zero;
    }
    vn = own < a.dv ? to_f32(vg[(size_t)t * a.dv + own]) : 0.f;
    bn = a.beta[(size_t)bh * a.T + t];
    ln = a.log_alpha[(size_t)bh * a.T + t];
  };
  load_token(0);
  // A row of the batch without a state of its own (a slot outside the pool, or one that an
  // earlier row of the batch names) writes no state and answers with zeros. The state's loads
  // do not wait for the search among the earlier rows.
  const int slot = a.slots ? a.slots[b] : b;
  bool live = slot >= 0 && slot < a.P;
  float* Sg = a.S + ((size_t)(live ? slot : 0) * a.H + h) * a.dv * dk;
  float4 s[kRows][NK4];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int i = 0; i < NK4; ++i)
      s[r][i] = live && nb + r < a.dv && kok[i]
                    ? load4(Sg + (size_t)(nb + r) * dk + 4 * (gl + LPR * i)) : zero;
  if (a.slots) {
    bool taken = false;
    for (int i = threadIdx.x; i < b; i += kWarps * 32) taken |= a.slots[i] == slot;
    live = !__syncthreads_or(taken) && live;
  }
  Tio* yg = static_cast<Tio*>(a.y) + (size_t)bh * a.T * a.dv;
  if (!live) {
    for (int t = 0; t < a.T; ++t)
      for (int r = gl; r < kRows && nb + r < a.dv; r += LPR) yg[(size_t)t * a.dv + nb + r] = from_f32<Tio>(0.f);
    return;
  }
  for (int t = 0; t < a.T; ++t) {
    float4 qv[NK4], kv[NK4];
    float kq = 0.f;
#pragma unroll
    for (int i = 0; i < NK4; ++i) {
      qv[i] = qn[i];
      kv[i] = kn[i];
      kq += qv[i].x * kv[i].x + qv[i].y * kv[i].y + qv[i].z * kv[i].z + qv[i].w * kv[i].w;
    }
    const float be = bn, la = ln;
    const bool reset = la < kResetLog;  // whatever the state held, NaN among it, is gone
    const float al = expf(la);
    const float vv = vn;
    if (t + 1 < a.T) load_token(t + 1);
    kq = group_sum<LPR>(kq);
    float p[2 * kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float pk = 0.f, pq = 0.f;
#pragma unroll
      for (int i = 0; i < NK4; ++i) {
        s[r][i] = reset ? zero
                        : make_float4(al * s[r][i].x, al * s[r][i].y, al * s[r][i].z, al * s[r][i].w);
        pk = fmaf(s[r][i].x, kv[i].x, pk);
        pq = fmaf(s[r][i].x, qv[i].x, pq);
        pk = fmaf(s[r][i].y, kv[i].y, pk);
        pq = fmaf(s[r][i].y, qv[i].y, pq);
        pk = fmaf(s[r][i].z, kv[i].z, pk);
        pq = fmaf(s[r][i].z, qv[i].z, pq);
        pk = fmaf(s[r][i].w, kv[i].w, pk);
        pq = fmaf(s[r][i].w, qv[i].w, pq);
      }
      p[r] = pk;
      p[kRows + r] = pq;
    }
#pragma unroll
    for (int m = kRows, o = kHalf; m >= 1; m >>= 1, o >>= 1) {
      const bool up = gl & o;
#pragma unroll
      for (int e = 0; e < m; ++e) {
        const float give = up ? p[e] : p[m + e];
        p[e] = (up ? p[m + e] : p[e]) + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
#pragma unroll
    for (int o = kSpread / 2; o > 0; o >>= 1) p[0] += __shfl_xor_sync(0xffffffffu, p[0], o);
    // lower lanes: c = beta (v - S'k); upper lanes: y = scale (S'q + c k.q)
    const float own_c = be * (vv - p[0]), c_low = __shfl_xor_sync(0xffffffffu, own_c, kHalf);
    if (gl >= kHalf && gl % kSpread == 0 && own < a.dv)
      yg[(size_t)t * a.dv + own] = from_f32<Tio>(a.scale * fmaf(c_low, kq, p[0]));
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float c = __shfl_sync(0xffffffffu, own_c, r * kSpread, LPR);
#pragma unroll
      for (int i = 0; i < NK4; ++i) {
        s[r][i].x = fmaf(c, kv[i].x, s[r][i].x);
        s[r][i].y = fmaf(c, kv[i].y, s[r][i].y);
        s[r][i].z = fmaf(c, kv[i].z, s[r][i].z);
        s[r][i].w = fmaf(c, kv[i].w, s[r][i].w);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int i = 0; i < NK4; ++i)
      if (nb + r < a.dv && kok[i])
        *reinterpret_cast<float4*>(Sg + (size_t)(nb + r) * dk + 4 * (gl + LPR * i)) = s[r][i];
}

template <typename Tio, int LPR, int NK4, int kRows>
void launch_rows(const StepArgs& a, int ctas, cudaStream_t st) {
  step_kernel<Tio, LPR, NK4, kRows><<<ctas, kWarps * 32, 0, st>>>(a);
  count_launch();
}
// 8 rows per lane group keep more loads in flight, once there are CTAs enough all the same: with
// 64 x 16 heads of 128 x 128 24.2 us against 24.8 us with 4 (float32, 3 tokens: 36.0 against
// 37.8 us), but 6.1 us against 5.6 us with 4 x 8 heads of 64 x 64 (5 tokens; caches flushed).
template <typename Tio, int LPR, int NK4>
void launch(const StepArgs& a, cudaStream_t st) {
  constexpr int rows = kWarps * (32 / LPR);  // per row of a lane group
  const int c4 = a.B * a.H * ((a.dv + 4 * rows - 1) / (4 * rows));
  constexpr int big = LPR >= 16 ? 8 : 4;
  const int c8 = a.B * a.H * ((a.dv + big * rows - 1) / (big * rows));
  if (c8 >= 148 * 16)
    launch_rows<Tio, LPR, NK4, big>(a, c8, st);
  else
    launch_rows<Tio, LPR, NK4, 4>(a, c4, st);
}

template <typename Tio>
cudaError_t launch_t(const StepArgs& a, cudaStream_t st) {
  if (a.dk <= 32)
    launch<Tio, 8, 1>(a, st);
  else if (a.dk <= 64)
    launch<Tio, 16, 1>(a, st);
  else if (a.dk <= 128)
    launch<Tio, 32, 1>(a, st);
  else
    launch<Tio, 32, 2>(a, st);
  return cudaGetLastError();
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

}  // namespace
}  // namespace delta
}  // namespace gradlev

using namespace gradlev;

extern "C" gradlev_status gradlev_delta_step(int B, int H, int Hk, int T, int d_k, int d_v,
                                             gradlev_dtype dt, const void* q, const void* k,
                                             const void* v, const float* beta,
                                             const float* log_alpha, float scale, const int* slots,
                                             int pool, float* S, void* y, void* stream) {
  using namespace gradlev::delta;
  reset_launch_count();
  if (B <= 0 || H <= 0 || Hk <= 0 || T <= 0 || d_k <= 0 || d_v <= 0 || pool <= 0)
    return GRADLEV_ERR_INVALID_ARG;
  if (dt != GRADLEV_F32 && dt != GRADLEV_BF16) return GRADLEV_ERR_INVALID_ARG;
  if (H % Hk != 0 || d_k % 4 != 0 || d_k > kMaxDk) return GRADLEV_ERR_UNSUPPORTED;
  const long long BH = (long long)B * H;  // the products of three may pass 64 bits
  if (BH >= 1LL << 31 || BH * T >= 1LL << 31 || BH * d_v >= 1LL << 30) return GRADLEV_ERR_UNSUPPORTED;
  if (!q || !k || !v || !beta || !log_alpha || !S || !y) return GRADLEV_ERR_INVALID_ARG;
  if (!slots && pool < B) return GRADLEV_ERR_INVALID_ARG;
  const size_t es = dt == GRADLEV_BF16 ? 2 : 4;
  if (!aligned(q, 4 * es) || !aligned(k, 4 * es) || !aligned(v, es) || !aligned(y, es) ||
      !aligned(beta, 4) || !aligned(log_alpha, 4) || !aligned(S, 16) || (slots && !aligned(slots, 4)))
    return GRADLEV_ERR_INVALID_ARG;
  const StepArgs a{B, H, Hk, T, d_k, d_v, pool, q, k, v, beta, log_alpha, scale, slots, S, y};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dt == GRADLEV_BF16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
  return e == cudaSuccess ? GRADLEV_OK : GRADLEV_ERR_CUDA;
}
