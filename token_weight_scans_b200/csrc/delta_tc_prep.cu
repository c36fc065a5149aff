// Tensor-core gated delta rule: the chunk-local matrices (delta_tc.h, struct Mats), one
// CTA per (chunk, value head), two CTAs per SM.
//
// K K^T and Q K^T go through the tensor core; the unit lower triangular inverse
// T0 = (I + A diag(beta))^-1 is formed in float32 by halves: 16 x 16 diagonal blocks by
// forward substitution (a lane per column, in registers), then twice
//   [[X1, 0], [-X2 N21 X1, X2]]
// which is as stable as substitution and needs only two products per level. The scaled
// matrices T0 diag(G), diag(w) T and P then multiply K (or T) on the tensor core; K is
// exact in bf16, so the gates ride on the other operand.
//
// beta = 0 leaves T0's column zero, but T's column j needs A's: columns are computed with
// beta at least 2^-60 in size, and T_ij = beta_i T0_ij / beta_j recovers them; T0 itself is
// off by 2^-60.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <atomic>

#include "delta_tc.h"
#include "sm100.cuh"

namespace gradlev {
namespace delta {
namespace tc {

using namespace sm100;

namespace {

constexpr int kThreads = 128;
constexpr int LD = 68;        // row stride (floats) of the 64 x 64 float32 matrices: 16-byte rows
constexpr int LT = 36;        // and of the 32 x 32 temporary
constexpr uint32_t COL_KQ = 0, COL_W = 64, kCols = 256;  // K K^T | Q K^T, then PT; W | Wb

struct PrepSmem {
  uint8_t K[2 * TILE], Q[2 * TILE];      // k-blocks: 64 token rows x 128 B
  uint8_t Tg[TILE], Tgl[TILE];           // T0 diag(G): bf16, and its remainder
  uint8_t Tw[TILE], Tt[TILE], P[TILE];   // diag(w) T, T, P
  float X[C * LD], N[C * LD];            // T0; A diag(beta)
  float tmp[32 * LT];
  float Lh[C], Ll[C], be[C], G[C], w[C];
  int seg[C];
  uint64_t full, mma;
  uint32_t tmem_base;
  int abort;
};
constexpr size_t kSmem = sizeof(PrepSmem) + 1024;
static_assert(2 * kSmem <= 227 * 1024, "two CTAs per SM");

enum : uint32_t { W_PREP_LOAD = 0x801, W_PREP_MMA };

struct PrepParams {
  Dims d;
  const float *beta, *log_alpha;
  float scale;
  DeviceStatus* status;
  uint64_t timeout_ns;
  Mats m;
  int split, back;   // remainders; Wb and PT
};

__device__ __forceinline__ uint32_t pack_lo(float a, float b, uint32_t hi) {
  return pack_bf16(a - bf16_lo(hi), b - bf16_hi(hi));
}

// D[r][c..c+7] (r = tid / 4 rows, 8 columns) = sum_m A[r][m] B[m][c], m < n
__device__ __forceinline__ void row8(float (&s)[8], const float* A, const float* B, int ldb, int n) {
#pragma unroll 4
  for (int m = 0; m < n; ++m) {
    const float a = A[m];
    const float4 b0 = *reinterpret_cast<const float4*>(B + m * ldb);
    const float4 b1 = *reinterpret_cast<const float4*>(B + m * ldb + 4);
    s[0] = fmaf(a, b0.x, s[0]);
    s[1] = fmaf(a, b0.y, s[1]);
    s[2] = fmaf(a, b0.z, s[2]);
    s[3] = fmaf(a, b0.w, s[3]);
    s[4] = fmaf(a, b1.x, s[4]);
    s[5] = fmaf(a, b1.y, s[5]);
    s[6] = fmaf(a, b1.z, s[6]);
    s[7] = fmaf(a, b1.w, s[7]);
  }
}

}  // namespace

__global__ void __launch_bounds__(kThreads) prep_kernel(const __grid_constant__ CUtensorMap tmK,
                                                        const __grid_constant__ CUtensorMap tmQ,
                                                        const __grid_constant__ CUtensorMap tmW,
                                                        const __grid_constant__ CUtensorMap tmWlo,
                                                        const __grid_constant__ CUtensorMap tmWb,
                                                        PrepParams p) {
  extern __shared__ uint8_t smem_raw[];
  PrepSmem& sm = *reinterpret_cast<PrepSmem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int N = chunks(p.d.T), bh = blockIdx.x / N, n = blockIdx.x - bh * N;
  const int b = bh / p.d.H, h = bh - b * p.d.H;
  const int kh = b * p.d.Hk + h / (p.d.H / p.d.Hk);
  const int t0 = n * C;
  const WaitCtx wc{&sm.abort, p.status, p.timeout_ns};
  if (tid == 0) {
    sm.abort = 0;
    mbar_init(&sm.full, 1);
    mbar_init(&sm.mma, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(&sm.full, 4 * TILE);
    tma_load_3d(sm.K, &tmK, &sm.full, 0, t0, kh);
    tma_load_3d(sm.K + TILE, &tmK, &sm.full, 64, t0, kh);
    tma_load_3d(sm.Q, &tmQ, &sm.full, 0, t0, kh);
    tma_load_3d(sm.Q + TILE, &tmQ, &sm.full, 64, t0, kh);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, kCols);
    tmem_relinquish();
  }
  if (warp == 2) {
    const GatePair g = chunk_gates(p.beta, p.log_alpha, (size_t)bh * p.d.T, t0, p.d.T);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = lane + 32 * k;
      sm.Lh[i] = g.Lh[k];
      sm.Ll[i] = g.Ll[k];
      sm.seg[i] = g.seg[k];
      sm.be[i] = g.be[k];
      sm.G[i] = gate_G(g, k);
      sm.w[i] = gate_w(g, k);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = sm.tmem_base;
  const uint32_t sK = smem_u32(sm.K), sQ = smem_u32(sm.Q);
  mbar_wait(&sm.full, 0, wc, W_PREP_LOAD);
  if (tid == 0) {
    const uint32_t id = idesc_bf16(64, 64, false, false);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const uint32_t off = (kk >> 2) * TILE + (kk & 3) * 32;
      const uint64_t dk = desc_at(sw128_desc(sK, 16, 1024), off);
      umma_bf16(tb + COL_KQ, dk, dk, id, kk > 0);
      umma_bf16(tb + COL_KQ + LANE16, desc_at(sw128_desc(sQ, 16, 1024), off), dk, id, kk > 0);
    }
    umma_commit(&sm.mma);
  }
  __syncwarp();
  mbar_wait(&sm.mma, 0, wc, W_PREP_MMA);
  __syncwarp();
  tc_fence_after();
  // Lane l < 16 of warp q holds row i = 16 q + l of K K^T, lane l + 16 that of Q K^T.
  const int i = 16 * warp + (lane & 15);
  const bool isP = lane >= 16;
  {
    const float Lh = sm.Lh[i], Ll = sm.Ll[i];
    const int seg = sm.seg[i];
    bf16* Pg = p.m.Pb + (((size_t)bh * N + n) * C + i) * C;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float v[32];
      tmem_ld32(tb + COL_KQ + ((uint32_t)(32 * warp) << 16) + 32 * half, v);
      tmem_ld_wait();
      uint32_t pp[16], pb[16];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        float x[2], xb[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int j = 32 * half + e + u;
          const bool on = (isP ? j <= i : j < i) && sm.seg[j] == seg;
          float be = sm.be[j];
          x[u] = on ? v[e + u] * expf((Lh - sm.Lh[j]) + (Ll - sm.Ll[j])) : 0.f;
          if (isP) {
            x[u] *= p.scale;
          } else {
            be = fabsf(be) < 0x1p-60f ? 0x1p-60f : be;
          }
          xb[u] = x[u] * be;
        }
        if (!isP) {
          *reinterpret_cast<float2*>(sm.N + i * LD + 32 * half + e) = make_float2(xb[0], xb[1]);
        }
        pp[e >> 1] = pack_bf16(x[0], x[1]);
        pb[e >> 1] = pack_bf16(xb[0], xb[1]);
      }
      if (isP) {
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          reinterpret_cast<uint4*>(Pg)[4 * half + cc] =
              make_uint4(pb[4 * cc], pb[4 * cc + 1], pb[4 * cc + 2], pb[4 * cc + 3]);
          if (p.back)
            st_shared_v4(smem_u32(sm.P) + sw128_off(i, 4 * half + cc), pp[4 * cc], pp[4 * cc + 1],
                         pp[4 * cc + 2], pp[4 * cc + 3]);
        }
      }
      __syncwarp();  // the next load is warp-collective
    }
  }
  tc_fence_before();
  __syncthreads();
  // ---- T0: 16 x 16 diagonal blocks, a lane per column
  {
    const int o = 16 * warp, c = lane & 15;
    float x[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float s = r == c ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < r; ++m) s = fmaf(-sm.N[(o + r) * LD + o + m], x[m], s);
      x[r] = s;
    }
    if (lane < 16) {
#pragma unroll
      for (int r = 0; r < 16; ++r) sm.X[(o + r) * LD + o + c] = x[r];
    } else {  // the blocks to the right of the diagonal
      for (int r = 0; r < 16; ++r)
        for (int cc = o + 16 + c; cc < C; cc += 16) sm.X[(o + r) * LD + cc] = 0.f;
    }
  }
  __syncthreads();
  // ---- 16 -> 32: two pairs of blocks, 64 threads each: row r, 4 columns
  {
    const int pr = tid >> 6, r = (tid & 63) >> 2, c = 4 * (tid & 3), o = 32 * pr;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < 16; ++m) {
      const float a = sm.N[(o + 16 + r) * LD + o + m];
      const float4 x = *reinterpret_cast<const float4*>(sm.X + (o + m) * LD + o + c);
      s[0] = fmaf(a, x.x, s[0]);
      s[1] = fmaf(a, x.y, s[1]);
      s[2] = fmaf(a, x.z, s[2]);
      s[3] = fmaf(a, x.w, s[3]);
    }
    *reinterpret_cast<float4*>(sm.tmp + (16 * pr + r) * LT + c) = make_float4(s[0], s[1], s[2], s[3]);
    __syncthreads();
    s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
    for (int m = 0; m < 16; ++m) {
      const float a = -sm.X[(o + 16 + r) * LD + o + 16 + m];
      const float4 x = *reinterpret_cast<const float4*>(sm.tmp + (16 * pr + m) * LT + c);
      s[0] = fmaf(a, x.x, s[0]);
      s[1] = fmaf(a, x.y, s[1]);
      s[2] = fmaf(a, x.z, s[2]);
      s[3] = fmaf(a, x.w, s[3]);
    }
    *reinterpret_cast<float4*>(sm.X + (o + 16 + r) * LD + o + c) = make_float4(s[0], s[1], s[2], s[3]);
  }
  __syncthreads();
  // ---- 32 -> 64: row r, 8 columns
  {
    const int r = tid >> 2, c = 8 * (tid & 3);
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    row8(s, sm.N + (32 + r) * LD, sm.X + c, LD, 32);
    float* t = sm.tmp + r * LT + c;
    *reinterpret_cast<float4*>(t) = make_float4(s[0], s[1], s[2], s[3]);
    *reinterpret_cast<float4*>(t + 4) = make_float4(s[4], s[5], s[6], s[7]);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.f;
    row8(s, sm.X + (32 + r) * LD + 32, sm.tmp + c, LT, 32);
    float* x = sm.X + (32 + r) * LD + c;
    *reinterpret_cast<float4*>(x) = make_float4(-s[0], -s[1], -s[2], -s[3]);
    *reinterpret_cast<float4*>(x + 4) = make_float4(-s[4], -s[5], -s[6], -s[7]);
  }
  __syncthreads();
  // ---- operands: thread (row r, 32 columns)
  {
    const int r = tid >> 1, c0 = 32 * (tid & 1);
    const size_t at = (((size_t)bh * N + n) * C + r) * C + c0;
    const float wr = sm.w[r], br = sm.be[r];
#pragma unroll
    for (int g = 0; g < 4; ++g) {  // 8 columns, one 16-byte piece
      uint32_t hi[4], lo[4], gh[4], gl[4], tw[4], tt[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = c0 + 8 * g + 2 * e;
        const float2 x = *reinterpret_cast<const float2*>(sm.X + r * LD + c);
        hi[e] = pack_bf16(x.x, x.y);
        lo[e] = pack_lo(x.x, x.y, hi[e]);
        const float ga = -x.x * sm.G[c], gb = -x.y * sm.G[c + 1];
        gh[e] = pack_bf16(ga, gb);
        gl[e] = pack_lo(ga, gb, gh[e]);
        if (p.back) {
          const float b0 = sm.be[c], b1 = sm.be[c + 1];
          const float ta = c < r ? br * x.x / (fabsf(b0) < 0x1p-60f ? 0x1p-60f : b0) : x.x;
          const float tbv = c + 1 < r ? br * x.y / (fabsf(b1) < 0x1p-60f ? 0x1p-60f : b1) : x.y;
          tw[e] = pack_bf16(wr * ta, wr * tbv);
          tt[e] = pack_bf16(ta, tbv);
        }
      }
      const uint32_t off = sw128_off(r, (c0 >> 3) + g);
      *reinterpret_cast<uint4*>(p.m.T0 + at + 8 * g) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      st_shared_v4(smem_u32(sm.Tg) + off, gh[0], gh[1], gh[2], gh[3]);
      if (p.split) {
        *reinterpret_cast<uint4*>(p.m.T0lo + at + 8 * g) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        st_shared_v4(smem_u32(sm.Tgl) + off, gl[0], gl[1], gl[2], gl[3]);
      }
      if (p.back) {
        st_shared_v4(smem_u32(sm.Tw) + off, tw[0], tw[1], tw[2], tw[3]);
        st_shared_v4(smem_u32(sm.Tt) + off, tt[0], tt[1], tt[2], tt[3]);
      }
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    tc_fence_after();
    const uint32_t id_w = idesc_bf16(64, 128, false, true), id_wb = idesc_bf16(64, 128, true, true);
    const uint32_t id_pt = idesc_bf16(64, 64, false, true);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const uint64_t dk = desc_at(sw128_desc(sK, TILE, 1024), kk * 2048);  // K as [token][d_k]
      umma_bf16(tb + COL_W, desc_at(sw128_desc(smem_u32(sm.Tg), 16, 1024), kk * 32), dk, id_w, kk > 0);
      if (p.split)
        umma_bf16(tb + COL_W, desc_at(sw128_desc(smem_u32(sm.Tgl), 16, 1024), kk * 32), dk, id_w, 1);
      if (p.back) {
        umma_bf16(tb + COL_W + LANE16, desc_at(sw128_desc(smem_u32(sm.Tw), TILE, 1024), kk * 2048),
                  dk, id_wb, kk > 0);
        umma_bf16(tb + COL_KQ, desc_at(sw128_desc(smem_u32(sm.P), 16, 1024), kk * 32),
                  desc_at(sw128_desc(smem_u32(sm.Tt), TILE, 1024), kk * 2048), id_pt, kk > 0);
      }
    }
    umma_commit(&sm.mma);
  }
  __syncwarp();
  mbar_wait(&sm.mma, 1, wc, W_PREP_MMA);
  __syncwarp();
  tc_fence_after();
  // W (lanes < 16) and Wb (lanes >= 16) to bf16; staged over Q (W), K (Wb) and the operand
  // tiles Tg, Tgl (the remainder of W), which every product has read
#pragma unroll
  for (int g = 0; g < 4; ++g) {  // 32 columns
    float v[32];
    tmem_ld32(tb + COL_W + ((uint32_t)(32 * warp) << 16) + 32 * g, v);
    tmem_ld_wait();
    const bool on = !isP || p.back;
    const uint32_t dst = smem_u32(isP ? sm.K : sm.Q) + (g >> 1) * TILE;
    const uint32_t dlo = smem_u32(sm.Tg) + (g >> 1) * TILE;  // Tg and Tgl are adjacent
#pragma unroll
    for (int cc = 0; cc < 4; ++cc) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        hi[e] = pack_bf16(v[8 * cc + 2 * e], v[8 * cc + 2 * e + 1]);
        lo[e] = pack_lo(v[8 * cc + 2 * e], v[8 * cc + 2 * e + 1], hi[e]);
      }
      const uint32_t off = sw128_off(i, 4 * (g & 1) + cc);
      if (on) st_shared_v4(dst + off, hi[0], hi[1], hi[2], hi[3]);
      if (p.split && !isP) st_shared_v4(dlo + off, lo[0], lo[1], lo[2], lo[3]);
    }
    __syncwarp();
  }
  if (p.back) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float v[32];
      tmem_ld32(tb + COL_KQ + ((uint32_t)(32 * warp) << 16) + 32 * half, v);
      tmem_ld_wait();
      if (!isP) {
        uint4* out = reinterpret_cast<uint4*>(p.m.PT + (((size_t)bh * N + n) * C + i) * C + 32 * half);
#pragma unroll
        for (int cc = 0; cc < 4; ++cc)
          out[cc] = make_uint4(pack_bf16(v[8 * cc], v[8 * cc + 1]), pack_bf16(v[8 * cc + 2], v[8 * cc + 3]),
                               pack_bf16(v[8 * cc + 4], v[8 * cc + 5]), pack_bf16(v[8 * cc + 6], v[8 * cc + 7]));
      }
      __syncwarp();
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    for (int kb = 0; kb < 2; ++kb) {
      tma_store_3d(&tmW, sm.Q + kb * TILE, 64 * kb, t0, bh);
      if (p.split) tma_store_3d(&tmWlo, sm.Tg + kb * TILE, 64 * kb, t0, bh);
      if (p.back) tma_store_3d(&tmWb, sm.K + kb * TILE, 64 * kb, t0, bh);
    }
    tma_store_commit();
    tma_store_wait_all();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tb, kCols);
  }
}

cudaError_t launch_prep(const Args& a, bool split, cudaStream_t st) {
  const Dims& d = a.d;
  const uint64_t N = chunks(d.T), kh = (uint64_t)d.B * d.Hk, bh = d.BH();
  const bool back = a.m.Wb != nullptr;
  CUtensorMap mk, mq, mw, mwl, mwb;
  using gradlev::tc::make_map_bf16_3d;
  if (!make_map_bf16_3d(&mk, a.k, 128, d.T, kh, C) || !make_map_bf16_3d(&mq, a.q, 128, d.T, kh, C) ||
      !make_map_bf16_3d(&mw, a.m.W, 128, N * C, bh, C) ||
      !make_map_bf16_3d(&mwl, split ? a.m.Wlo : a.m.W, 128, N * C, bh, C) ||
      !make_map_bf16_3d(&mwb, back ? a.m.Wb : a.m.W, 128, N * C, bh, C))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!bit || !(set.load() & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit);
  }
  PrepParams p{d, a.beta, a.log_alpha, a.scale, a.status, a.timeout_ns, a.m, split, back};
  prep_kernel<<<(unsigned)(N * bh), kThreads, kSmem, st>>>(mk, mq, mw, mwl, mwb, p);
  count_launch();
  return cudaGetLastError();
}

}  // namespace tc
}  // namespace delta
}  // namespace gradlev
