// Tensor-core gated delta rule: the chunk-local matrices (delta_tc.h, struct Mats) of one
// (chunk, value head) after the other, three persistent CTAs per SM (two with THREE).
//
// K K^T and Q K^T go through the tensor core; the unit lower triangular inverse
// T0 = (I + A diag(beta))^-1 is formed in float32 by halves: 16 x 16 diagonal blocks by
// forward substitution (a lane per column, in registers), then twice
//   [[X1, 0], [-X2 N21 X1, X2]]
// which is as stable as substitution and needs only two products per level (warp-wide tf32
// products of split operands: float32 FMAs took 25 us more of a B8 H16 T4096, their shared-memory
// reads held the kernel up; tiles this small leave tcgen05.mma idle).
//
// Kw = T0^T diag(beta w) K, Pv = P diag(beta) T0 and Wq = scale diag(G) Q - Pv diag(G) K then go
// through the tensor core again. Their terms cancel where keys are alike, so T0, P and Pv diag(G)
// enter as two bf16 each (K is exact in bf16): the results are good to 2^-16 before they are
// rounded.
//
// beta = 0 would leave T0's column zero where E's row needs it: beta is taken at least 2^-60 in
// size here (bt), which puts T0, Pv and Kw off by no more than that.
//
// Measured (B8 H16 T4096 d 128, 8192 chunks): 313 us with the backward's matrices, 2110 bytes per
// token or 3.5 TB/s; 395 us with Kw in three parts in place of those (B1 H16 T32768, two CTAs per
// SM). What bounds it is the chain of short steps through a chunk at 24 warps per SM: 35 % of the issue
// slots, 30 % of the shared-memory pipe, 19 % of the tensor pipe, 30 % of the DRAM. Registers decide:
// products unrolled over their terms spill. (W = -T0 diag(G) K and P diag(beta) for an unfolded
// form, in one bf16 each, took 185 us.)
//
// Waits: the in-flight TMA stores only read shared memory, so the CTA waits for that read
// and not for their completion; the end of the kernel, which the walk waits for, orders them.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <atomic>

#include "delta_tc.h"
#include "sm100.cuh"
#include "tf32.cuh"

namespace gradlev {
namespace delta {
namespace tc {

using namespace sm100;

namespace {

constexpr int kThreads = 256;
constexpr int LD = 68;        // row stride (floats) of the 64 x 64 float32 matrices: 16-byte rows
// TMEM, in the lower and the upper 16 lanes of each 32: K K^T | Q K^T (64 columns); Kw | Pv (64);
// Kw | Wq
constexpr uint32_t kCols = 128;
constexpr float kTiny = 0x1p-60f;
constexpr int kLoader = 128;  // the thread that loads K and Q, and stores P and PT

// Tiles live where something dead was. Over N: diag(beta w) T0, then Pv diag(G), at the end Kw. Over
// X: T0, then Pv, at the end the remainder of Kw. Over Q: P diag(beta) (all these two bf16 each);
// then Q again, from L2, and Wq over it, row by row as it is formed, with BACK its remainder over K.
// THREE has a place for the third part of diag(beta w) T0, and then of Kw.
template <bool THREE>
struct PrepSmem {
  uint8_t K[2 * TILE];         // k-blocks: 64 token rows x 128 B
  uint8_t Q[2 * TILE];
  union {
    float N[C * LD];           // A diag(beta); parts that are done with hold the products' halves
    uint8_t A[2][TILE];
  };
  union {
    float X[C * LD];           // T0
    uint8_t B[2][TILE];
  };
  alignas(1024) uint8_t Z[THREE ? 2 * TILE : 16];
  // per token: M_ij = ra_i ca_j with both factors within e^40 (fac: all decays of the chunk within
  // e^80, and the factors taken from the middle of that range, so that ca kTiny stays a normal
  // number: a factor taken from a token, e^-80 kTiny, would underflow and take dbeta with it where
  // beta = 0); bt is beta, at least kTiny in size: cb = ca bt, wb = w bt, sG = scale G
  float ra[C], cb[C];
  float Lh[C], Ll[C], G[C], wb[C], sG[C];
  int seg[C];
  int fac;
  uint64_t full, qfull, mma;
  uint32_t tmem_base;
  int abort;
};
template <bool THREE> constexpr size_t smem_bytes() { return sizeof(PrepSmem<THREE>) + 1024; }
static_assert(3 * (smem_bytes<false>() + 1024) <= 228 * 1024, "three CTAs per SM");
static_assert(2 * (smem_bytes<true>() + 1024) <= 228 * 1024, "two CTAs per SM");

enum : uint32_t { W_PREP_LOAD = 0x801, W_PREP_Q, W_PREP_MMA, W_PREP_DRAIN };

struct PrepParams {
  Dims d;
  const float *beta, *log_alpha;
  float scale;
  DeviceStatus* status;
  uint64_t timeout_ns;
  Mats m;
};

__device__ __forceinline__ uint32_t pack_lo(float a, float b, uint32_t hi) {
  return pack_bf16(a - bf16_lo(hi), b - bf16_hi(hi));
}
__device__ __forceinline__ float4 at4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// 16 x 8 of a product of float32 matrices in shared memory (row stride LD), k0 <= k < k1 (whole
// eights): out[0..1] in row lane / 4, out[2..3] eight rows below, at columns 2 (lane % 4) and the
// next.
__device__ __forceinline__ void product16x8(float (&out)[4], const float* A, const float* B, int k0,
                                            int k1) {
  out[0] = out[1] = out[2] = out[3] = 0.f;
  tf32::tile<false>(out, k0, k1, [&](int r, int k) { return A[r * LD + k]; },
                    [&](int k, int c) { return B[k * LD + c]; });
}
__device__ __forceinline__ void store16x8(float* at, const float (&v)[4], float sign) {
  float* p = at + ((threadIdx.x & 31) >> 2) * LD + 2 * (threadIdx.x & 3);
  *reinterpret_cast<float2*>(p) = make_float2(sign * v[0], sign * v[1]);
  *reinterpret_cast<float2*>(p + 8 * LD) = make_float2(sign * v[2], sign * v[3]);
}

}  // namespace

// THREE: Kw in three parts; BACK: T0 and the remainder of Wq, for the backward.
template <bool THREE, bool BACK>
__global__ void __launch_bounds__(kThreads, THREE ? 2 : 3)
    prep_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                const __grid_constant__ CUtensorMap tmKw, const __grid_constant__ CUtensorMap tmKw2,
                const __grid_constant__ CUtensorMap tmKw3, const __grid_constant__ CUtensorMap tmWq,
                const __grid_constant__ CUtensorMap tmWq2, const __grid_constant__ CUtensorMap tmPv,
                PrepParams p) {
  extern __shared__ uint8_t smem_raw[];
  using Smem = PrepSmem<THREE>;
  Smem& sm = *reinterpret_cast<Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int N = chunks(p.d.T);
  const WaitCtx wc{&sm.abort, p.status, p.timeout_ns};
  const unsigned total = (unsigned)((size_t)p.d.B * p.d.H * N);
  // one thread: K or Q of a chunk
  auto load = [&](unsigned id, bool q, uint64_t* bar) {
    const int bh = id / N, t0 = (id - bh * N) * C, b = bh / p.d.H, h = bh - b * p.d.H;
    const int kh = b * p.d.Hk + h / (p.d.H / p.d.Hk);
    tma_load_3d(q ? sm.Q : sm.K, q ? &tmQ : &tmK, bar, 0, t0, kh);
    tma_load_3d((q ? sm.Q : sm.K) + TILE, q ? &tmQ : &tmK, bar, 64, t0, kh);
  };
  grid_dep_launch();
  RawGates raw{};
  auto load_raw = [&](unsigned id) {  // warp 2
    const int bh = id / N;
    raw = load_gates(p.beta, p.log_alpha, (size_t)bh * p.d.T, (id - bh * N) * C, p.d.T);
  };
  if (warp == 2) load_raw(blockIdx.x);
  if (tid == kLoader) {
    sm.abort = 0;
    mbar_init(&sm.full, 1);
    mbar_init(&sm.qfull, 1);
    mbar_init(&sm.mma, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(&sm.full, 4 * TILE);
    load(blockIdx.x, false, &sm.full);
    load(blockIdx.x, true, &sm.full);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = sm.tmem_base;
  const uint32_t sK = smem_u32(sm.K), sQ = smem_u32(sm.Q), sA = smem_u32(sm.A[0]), sB = smem_u32(sm.B[0]);
  const uint32_t sZ = smem_u32(sm.Z);
  uint32_t phase = 0, full = 0, loads = 0, again = 0;  // loads after the first, and of Q again (loading thread)
  for (unsigned id = blockIdx.x; id < total; id += gridDim.x, full ^= 1) {
  const int bh = id / N, n = id - bh * N, t0 = n * C;
  if (tid == 0) {
    mbar_wait(&sm.full, full, wc, W_PREP_LOAD);
    tc_fence_after();
    const uint32_t id = idesc_bf16(64, 64, false, false);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const uint32_t off = (kk >> 2) * TILE + (kk & 3) * 32;
      const uint64_t dk = desc_at(sw128_desc(sK, 16, 1024), off);
      umma_bf16(tb, dk, dk, id, kk > 0);
      umma_bf16(tb + LANE16, desc_at(sw128_desc(sQ, 16, 1024), off), dk, id, kk > 0);
    }
    umma_commit(&sm.mma);
  }
  __syncwarp();
  if (warp == 2) {
    const GatePair g = chunk_gates(raw);
    if (id + gridDim.x < total) load_raw(id + gridDim.x);
    const float Lm = 0.5f * g.Lend, Ll = 0.5f * g.Lend_lo;
    const bool fac = g.seg_end == 0 && g.Lend > -80.f;
    GateBlock* gb = reinterpret_cast<GateBlock*>(p.m.gates) + (size_t)bh * N + n;
    if (lane == 0) {
      gb->GC = gb->GCb = gate_GC(g);
      gb->fac = fac ? 1.f : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = lane + 32 * k;
      const float be = g.be[k], bt = fabsf(be) < kTiny ? kTiny : be;
      const float x = (g.Lh[k] - Lm) + (g.Ll[k] - Ll);
      const float ca = fac ? expf(-x) : 1.f;
      sm.ra[i] = fac ? expf(x) : 1.f;
      sm.cb[i] = ca * bt;
      sm.Lh[i] = g.Lh[k];
      sm.Ll[i] = g.Ll[k];
      sm.seg[i] = g.seg[k];
      const float G = gate_G(g, k), w = gate_w(g, k), z = fabsf(be) < kTiny ? be / bt : 1.f;
      sm.G[i] = G;
      sm.sG[i] = p.scale * G;
      sm.wb[i] = w * bt;
      gb->nG[i] = -G;
      gb->z[i] = gb->zb[i] = z;
      gb->zG[i] = -G * z;
      gb->rb[i] = 1.f / bt;
      gb->bw[i] = be * w;
      gb->q[i] = p.scale * G;
      gb->bG[i] = -be * G;
      gb->be[i] = be;
      gb->ra[i] = sm.ra[i];
      gb->cb[i] = ca * be;
    }
    if (lane == 0) sm.fac = fac;
  }
  mbar_wait(&sm.mma, phase, wc, W_PREP_MMA);
  phase ^= 1;
  __syncthreads();  // the gates are there
  tc_fence_after();
  // Lane l < 16 of quadrant q holds row i = 16 q + l of K K^T, lane l + 16 that of Q K^T;
  // warps q and q + 4 take half of the columns each.
  const int q = warp & 3, hh = warp >> 2;
  const uint32_t lo = (uint32_t)(32 * q) << 16;
  const int i = 16 * q + (lane & 15);
  const bool isP = lane >= 16;
  // this thread's half row of K K^T or Q K^T, times M and bt (and scale), on and below the diagonal
  auto scaled = [&](float (&v)[32]) {
    tmem_ld32(tb + lo + 32 * hh, v);
    tmem_ld_wait();
    // the entries below (P: and on) the diagonal
    const int keep = i - 32 * hh + (isP ? 1 : 0);
    const float sc = isP ? p.scale : 1.f;
    if (sm.fac) {
      const float ra = sc * sm.ra[i];
      const float* cv = sm.cb + 32 * hh;
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 c = at4(cv + e);
        v[e] = e < keep ? v[e] * (ra * c.x) : 0.f;
        v[e + 1] = e + 1 < keep ? v[e + 1] * (ra * c.y) : 0.f;
        v[e + 2] = e + 2 < keep ? v[e + 2] * (ra * c.z) : 0.f;
        v[e + 3] = e + 3 < keep ? v[e + 3] * (ra * c.w) : 0.f;
      }
    } else {  // a reset, or decays whose factors leave float32
      const float Lh = sm.Lh[i], Ll = sm.Ll[i];
      const int seg = sm.seg[i];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int j = 32 * hh + e;
        const float m = sc * sm.cb[j] * expf(fminf((Lh - sm.Lh[j]) + (Ll - sm.Ll[j]), 0.f));
        v[e] = e < keep && sm.seg[j] == seg ? v[e] * m : 0.f;
      }
    }
  };
  // 32 columns of row i as two bf16 into a pair of tiles
  auto put_split = [&](uint32_t at, const float (&v)[32]) {
#pragma unroll
    for (int cc = 0; cc < 4; ++cc) {
      uint32_t hi[4], low[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        hi[e] = pack_bf16(v[8 * cc + 2 * e], v[8 * cc + 2 * e + 1]);
        low[e] = pack_lo(v[8 * cc + 2 * e], v[8 * cc + 2 * e + 1], hi[e]);
      }
      const uint32_t off = sw128_off(i, 4 * hh + cc);
      st_shared_v4(at + off, hi[0], hi[1], hi[2], hi[3]);
      st_shared_v4(at + TILE + off, low[0], low[1], low[2], low[3]);
    }
  };
  {
    float v[32];
    scaled(v);
    if (!isP) {
#pragma unroll
      for (int e = 0; e < 32; e += 4)
        *reinterpret_cast<float4*>(sm.N + i * LD + 32 * hh + e) =
            make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    } else {
      put_split(sQ, v);
    }
  }
  __syncthreads();
  // ---- T0: 16 x 16 diagonal blocks, two per warp, a lane per column; other warps clear what
  //      is right of them
  if (warp < 2) {
    const int o = 32 * warp + (lane & 16), c = lane & 15;
    float x[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float s = r == c ? 1.f : 0.f;
      const float* Nr = sm.N + (o + r) * LD + o;
#pragma unroll
      for (int m = 0; m < r; m += 4) {
        const float4 a = at4(Nr + m);
        s = fmaf(-a.x, x[m], s);
        if (m + 1 < r) s = fmaf(-a.y, x[m + 1], s);
        if (m + 2 < r) s = fmaf(-a.z, x[m + 2], s);
        if (m + 3 < r) s = fmaf(-a.w, x[m + 3], s);
      }
      x[r] = s;
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) sm.X[(o + r) * LD + o + c] = x[r];
  } else if (warp >= 4) {
    const int r = (tid - 128) >> 1, c1 = 32 * (tid & 1);  // row r, 32 columns
    for (int c = max(c1, (r & ~15) + 16); c < c1 + 32; c += 4)
      *reinterpret_cast<float4*>(sm.X + r * LD + c) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  // ---- 16 -> 32: two pairs of blocks, a warp for 8 columns of one. N21 X1 goes into the first
  //      diagonal block of N, done with; X1 is zero above its diagonal
  float s4[4];
  if (warp < 4) {
    const int o = 32 * (warp >> 1), c = 8 * (warp & 1);
    float* tmp = sm.N + o * LD + o + c;
    product16x8(s4, sm.N + (o + 16) * LD + o, sm.X + o * LD + o + c, c, 16);
    store16x8(tmp, s4, 1.f);
    __syncwarp();
    product16x8(s4, sm.X + (o + 16) * LD + o + 16, tmp, 0, 16);
    store16x8(sm.X + (o + 16) * LD + o + c, s4, -1.f);
  }
  __syncthreads();
  // ---- 32 -> 64, the same with two warps, of 16 rows each, for 8 columns
  {
    const int c = 8 * (warp >> 1), r = 16 * (warp & 1);
    product16x8(s4, sm.N + (32 + r) * LD, sm.X + c, c, 32);
    store16x8(sm.N + r * LD + c, s4, 1.f);
    asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp >> 1)) : "memory");
    product16x8(s4, sm.X + (32 + r) * LD + 32, sm.N + c, 0, r + 16);
    store16x8(sm.X + (32 + r) * LD + c, s4, -1.f);
  }
  __syncthreads();
  // ---- operands: a lane takes 8 columns of two rows, 8 lanes a row. Lanes 4 to 7 load their
  //      second half first, so that the loads have no bank conflicts.
  {
    const int c = 8 * (tid & 7), sw = tid & 4;
    auto at8 = [&](const float* p, float (&x)[8]) {
      const float4 a = at4(p + sw), b = at4(p + (4 - sw));
      x[0] = sw ? b.x : a.x, x[1] = sw ? b.y : a.y, x[2] = sw ? b.z : a.z, x[3] = sw ? b.w : a.w;
      x[4] = sw ? a.x : b.x, x[5] = sw ? a.y : b.y, x[6] = sw ? a.z : b.z, x[7] = sw ? a.w : b.w;
    };
    auto pack8 = [&](const float (&x)[8]) {
      return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                        pack_bf16(x[6], x[7]));
    };
    auto rest8 = [&](const float (&x)[8], const uint4& h) {
      return make_uint4(pack_lo(x[0], x[1], h.x), pack_lo(x[2], x[3], h.y), pack_lo(x[4], x[5], h.z),
                        pack_lo(x[6], x[7], h.w));
    };
    auto put = [&](uint32_t dst, const uint4& v) { st_shared_v4(dst, v.x, v.y, v.z, v.w); };
    uint4 hi[2], rest[2];
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const int r = (tid >> 3) + 32 * rr;
      float x[8];
      at8(sm.X + r * LD + c, x);
      hi[rr] = pack8(x);
      rest[rr] = rest8(x, hi[rr]);
      const float wr = sm.wb[r];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= wr;
      const uint32_t off = sw128_off(r, c >> 3);
      const uint4 h = pack8(x);
      const uint4 l = rest8(x, h);
      put(sA + off, h);
      put(sA + TILE + off, l);
      if (THREE) {
        const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] -= bf16_lo(hw[e]);
          x[2 * e + 1] -= bf16_hi(hw[e]);
        }
        put(sZ + off, rest8(x, l));
      }
    }
    __syncthreads();  // X is read, and T0 goes over it
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      const int r = (tid >> 3) + 32 * rr;
      const uint32_t off = sw128_off(r, c >> 3);
      put(sB + off, hi[rr]);
      put(sB + TILE + off, rest[rr]);
      if (BACK) {
        bf16* const at = p.m.T0 + (((size_t)bh * N + n) * C + r) * 128 + c;
        *reinterpret_cast<uint4*>(at) = hi[rr];
        *reinterpret_cast<uint4*>(at + 64) = rest[rr];
      }
    }
  }
  // One group of products of M = 64: d (+)= a b over the 64 tokens, from thread 0
  auto product = [&](uint32_t d, uint32_t a, bool a_mn, uint32_t b, int cols, bool first) {
    const uint32_t what = idesc_bf16(64, cols, a_mn, true);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      umma_bf16(d, a_mn ? desc_at(sw128_desc(a, TILE, 1024), kk * 2048)
                        : desc_at(sw128_desc(a, 16, 1024), kk * 32),
                desc_at(sw128_desc(b, TILE, 1024), kk * 2048), what, !first || kk > 0);
  };
  const uint32_t tU = tb + LANE16;  // the upper lanes
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {  // Kw and Pv
    tc_fence_after();
    product(tb, sA, true, sK, 128, true);
    product(tb, sA + TILE, true, sK, 128, false);
    if (THREE) product(tb, sZ, true, sK, 128, false);
    product(tU, sQ, false, sB, 64, true);
    product(tU, sQ, false, sB + TILE, 64, false);
    product(tU, sQ + TILE, false, sB, 64, false);
    umma_commit(&sm.mma);
  }
  __syncwarp();
  {
    const bool got = mbar_wait(&sm.mma, phase, wc, W_PREP_MMA);
    if (tid == kLoader && got) {
      mbar_arrive_expect_tx(&sm.qfull, 2 * TILE);
      load(id, true, &sm.qfull);
      ++again;
    }
  }
  phase ^= 1;
  __syncwarp();
  tc_fence_after();
  {
    float v[32];
    tmem_ld32(tb + lo + 32 * hh, v);
    tmem_ld_wait();
    if (isP) {
      put_split(sB, v);
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 g = at4(sm.G + 32 * hh + e);
        v[e] *= -g.x;
        v[e + 1] *= -g.y;
        v[e + 2] *= -g.z;
        v[e + 3] *= -g.w;
      }
      put_split(sA, v);
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  if (tid == kLoader) {
    tma_store_3d(&tmPv, sm.B[0], 0, t0, bh);
    tma_store_3d(&tmPv, sm.B[1], 64, t0, bh);
    tma_store_commit();
  }
  if (tid == 0) {  // - Pv diag(G) K
    tc_fence_after();
    product(tU, sA, false, sK, 128, true);
    product(tU, sA + TILE, false, sK, 128, false);
    umma_commit(&sm.mma);
  }
  __syncwarp();
  const bool done = mbar_wait(&sm.mma, phase, wc, W_PREP_MMA);
  phase ^= 1;
  const bool more = done && id + gridDim.x < total;
  if (tid == kLoader) {
    if (more) {
      mbar_arrive_expect_tx(&sm.full, 4 * TILE);
      if (!BACK) load(id + gridDim.x, false, &sm.full);
      ++loads;
    }
    tma_store_wait_read();  // Pv
  }
  mbar_wait(&sm.qfull, full, wc, W_PREP_Q);
  __syncthreads();
  tc_fence_after();
  // Kw (lanes < 16) and Wq (lanes >= 16) to bf16, columns [64 hh, 64 hh + 64)
  const float sG = sm.sG[i];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    float v[32];
    tmem_ld32(tb + lo + 64 * hh + 32 * g, v);
    tmem_ld_wait();
    const uint32_t dst = (isP ? sQ : sA) + hh * TILE;
#pragma unroll
    for (int cc = 0; cc < 4; ++cc) {
      const uint32_t off = sw128_off(i, 4 * g + cc);
      if (isP) {
        const uint4 u = ld_shared_v4(dst + off);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[8 * cc + 2 * e] = fmaf(sG, bf16_lo(w[e]), v[8 * cc + 2 * e]);
          v[8 * cc + 2 * e + 1] = fmaf(sG, bf16_hi(w[e]), v[8 * cc + 2 * e + 1]);
        }
      }
#pragma unroll
      for (int k = 0; k < (THREE ? 3 : 2); ++k) {  // the parts of Kw; of Wq one, or two
        uint32_t part[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float &a = v[8 * cc + 2 * e], &b = v[8 * cc + 2 * e + 1];
          part[e] = pack_bf16(a, b);
          a -= bf16_lo(part[e]);
          b -= bf16_hi(part[e]);
        }
        const uint32_t at = k == 0 ? dst : (k == 2 ? sZ : isP ? sK : sB) + hh * TILE;
        if (k == 0 || !isP || (BACK && k == 1)) st_shared_v4(at + off, part[0], part[1], part[2], part[3]);
      }
    }
    __syncwarp();
  }
  fence_proxy_async_smem();
  tc_fence_before();
  const bool stop = __syncthreads_or(*reinterpret_cast<volatile int*>(&sm.abort));
  if (tid == kLoader) {
    for (int kb = 0; kb < 2; ++kb) {
      tma_store_3d(&tmWq, sm.Q + kb * TILE, 64 * kb, t0, bh);
      tma_store_3d(&tmKw, sm.A[kb], 64 * kb, t0, bh);
      tma_store_3d(&tmKw2, sm.B[kb], 64 * kb, t0, bh);
      if (BACK) tma_store_3d(&tmWq2, sm.K + kb * TILE, 64 * kb, t0, bh);
      if (THREE) tma_store_3d(&tmKw3, sm.Z + kb * TILE, 64 * kb, t0, bh);
    }
    tma_store_commit();
    tma_store_wait_read();  // the places are written again from here on
    if (more && BACK) load(id + gridDim.x, false, &sm.full);
    if (more) load(id + gridDim.x, true, &sm.full);
  }
  __syncwarp();
  if (stop) break;
  }
  if (tid == kLoader) {
    mbar_drain(&sm.full, loads & 1, wc, W_PREP_DRAIN);
    if (again) mbar_drain(&sm.qfull, (again - 1) & 1, wc, W_PREP_DRAIN);
    tma_store_wait_read();  // shared memory may go once it is read
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tb, kCols);
  }
}

template <bool THREE, bool BACK>
static cudaError_t launch(const CUtensorMap (&m)[8], const PrepParams& p, unsigned grid, cudaStream_t st) {
  static std::atomic<uint64_t> set{0};  // devices whose opt-in is done
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!bit || !(set.load() & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(prep_kernel<THREE, BACK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem_bytes<THREE>());
    if (e != cudaSuccess) return e;
    set.fetch_or(bit);
  }
  const unsigned most = 148 * (THREE ? 2 : 3);
  prep_kernel<THREE, BACK><<<grid < most ? grid : most, kThreads, smem_bytes<THREE>(), st>>>(
      m[0], m[1], m[2], m[3], m[4], m[5], m[6], m[7], p);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_prep(const Args& a, bool last_state, cudaStream_t st) {
  const Dims& d = a.d;
  const uint64_t N = chunks(d.T), kh = (uint64_t)d.B * d.Hk, bh = d.BH();
  const bool back = a.m.T0 != nullptr;
  CUtensorMap m[8];
  using gradlev::tc::make_map_bf16_3d;
  auto mat = [&](CUtensorMap* t, const bf16* x) { return make_map_bf16_3d(t, x, 128, N * C, bh, C); };
  if (!make_map_bf16_3d(&m[0], a.k, d.dk, d.T, kh, C) || !make_map_bf16_3d(&m[1], a.q, d.dk, d.T, kh, C) ||
      !mat(&m[2], a.m.Kw) || !mat(&m[3], a.m.Kw2) || !mat(&m[4], a.m.Kw3) || !mat(&m[5], a.m.Wq) ||
      !mat(&m[6], back ? a.m.Wq2 : a.m.Wq) || !mat(&m[7], a.m.Pv))
    return cudaErrorInvalidValue;
  const PrepParams p{d, a.beta, a.log_alpha, a.scale, a.status, a.timeout_ns, a.m};
  const unsigned grid = (unsigned)(N * bh);
  if (last_state) return back ? launch<true, true>(m, p, grid, st) : launch<true, false>(m, p, grid, st);
  return back ? launch<false, true>(m, p, grid, st) : launch<false, false>(m, p, grid, st);
}

}  // namespace tc
}  // namespace delta
}  // namespace gradlev
