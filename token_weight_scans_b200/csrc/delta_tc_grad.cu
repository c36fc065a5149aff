// Tensor-core gated delta rule: the gradients of q, k and the gates of one chunk of 64
// tokens and one key head, from the states at the chunk's start, their gradients at its
// end, D and E (delta.h); two persistent CTAs per SM. The value heads that share the key head are
// taken in turn and add up in registers, so nothing is added through memory.
//
// Products of one value head (M = 64 tokens each; two share their TMEM columns, one in the
// lower and one in the upper 16 lanes of each 32):
//   F = dY D^T, H = E D^T (contracted over d_v)       t = dY S, u = E S, z = D dS
//   X = scale M beta_j F,  Yn = -M beta_i beta_j H
//   xk = X K,  yk = Yn K,  ka = X^T Q + Yn^T K
//   dQ += scale G t + xk,  dK += -beta G u + beta w z + ka + yk
// The pairs' share of dlog_alpha needs only row and column sums of X q.k - Y k.k, which
// are dot products of q and k with xk, yk and ka:
//   row - column = q.xk + k.yk - k.ka.
// Row and column sums come from the same X and Yn, so the parts that cancel over a
// range of tokens do so to float32 rounding.
// D, E, X and Yn are two bf16 each: their terms cancel in all of these sums where keys are alike.
// With one bf16 in their place dq and dk are 1 %, dlog_alpha 4 to 90 % off there.
//
// Measured: 389 us for B8 H16 T4096 d 128 (3352 bytes per token: 4.5 TB/s), 583 us for B1 H16
// T32768 d_v 256 (5632 bytes: 5.1 TB/s), 393 us where four heads share a key head. 43 % of the
// tensor pipe (M = 64 products run at half its rate; the remainders doubled their number), 36 % of
// the issue slots. Shared memory holds two CTAs, which leaves next to no L1, so that a spilled
// register costs a trip to L2: 300 bytes of spills per thread cost 20 us. Hence X and Yn one
// after the other in pieces, the sums that begin late, and float32 pairs (half the FMAs). The remainders of D and E
// leave no room for X and Yn beside them, so the next D and E are loaded when those are done with.
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

constexpr int kThreads = 256;
constexpr uint32_t kCols = 256;
constexpr uint32_t COL_A = 0;     // t | u, then . | yk
constexpr uint32_t COL_B = 128;   // F, H (64 columns each) | z, then xk | ka

struct GradGates {                           // GC .. cb of GateBlock
  float GC, fac, pad[2], bw[C], q[C], bG[C], be[C], ra[C], cb[C];
  static constexpr size_t offset = offsetof(GateBlock, GC);
};
static_assert(sizeof(GradGates) % 16 == 0 && GradGates::offset % 16 == 0 &&
              GradGates::offset + sizeof(GradGates) == offsetof(GateBlock, GCb), "a bulk copy");

struct GradSmem {
  uint8_t Q[2 * TILE], K[2 * TILE];          // k-blocks; at the end dq and dk
  uint8_t O[TILE];                           // dY: 64 tokens x 64 columns of d_v
  uint8_t S[2 * TILE], dS[2 * TILE];         // 64 rows of d_v x 128
  // D^T, E^T: 64 rows of d_v x 64 tokens, with their remainders; once the products of the last
  // slice have read them, X and Yn
  uint8_t D[2 * TILE], E[2 * TILE];
  GradGates gates[2];                        // this head's and the next one's
  float Lh[C], Ll[C];                        // where a reset or strong decays rule out g.fac
  int seg[C];
  float xs[2][C], ps[2][C], zs[2][C];        // per column half
  float red[8];
  uint64_t kq, full, de, mma;
  uint32_t tmem_base;
  int abort;
};
constexpr size_t kSmem = sizeof(GradSmem) + 1024;
static_assert(2 * kSmem <= 227 * 1024, "two CTAs per SM");

enum : uint32_t { W_G_KQ = 0xa01, W_G_FULL, W_G_DE, W_G_MMA, W_G_DRAIN };

struct GradParams {
  Dims d;
  const float *beta, *log_alpha, *gates;
  float scale;
  DeviceStatus* status;
  uint64_t timeout_ns;
  bf16 *dbeta, *dlog_alpha;
};

// Two float32 products at once.
struct F2 { unsigned long long v; };
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void get2(const F2& x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ F2 fma2(const F2& a, const F2& b, const F2& c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add2(const F2& a, const F2& b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// 8 columns of a swizzled bf16 row
__device__ __forceinline__ void row8(float (&x)[8], const uint8_t* tile, int r, int c8) {
  const uint4 u = *reinterpret_cast<const uint4*>(tile + sw128_off(r, c8));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = bf16_lo(w[e]);
    x[2 * e + 1] = bf16_hi(w[e]);
  }
}

// 8 values as two bf16 each, into a pair of tiles
__device__ __forceinline__ void put_split8(uint32_t at, const float* x) {
  uint32_t hi[4], rest[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    hi[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
    rest[e] = pack_bf16(x[2 * e] - bf16_lo(hi[e]), x[2 * e + 1] - bf16_hi(hi[e]));
  }
  st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
  st_shared_v4(at + TILE, rest[0], rest[1], rest[2], rest[3]);
}

__device__ __forceinline__ void tmem_ld(uint32_t at, float (&v)[8]) { tmem_ld8(at, v); }
__device__ __forceinline__ void tmem_ld(uint32_t at, float (&v)[16]) { tmem_ld16(at, v); }

}  // namespace

// GROUP: several value heads share a key head, and the sums in acc live across their products;
// without, they begin after the state's products, which spares the registers until then.
template <bool GROUP>
__global__ void __launch_bounds__(kThreads, 2)
    grad_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmD,
                const __grid_constant__ CUtensorMap tmE, const __grid_constant__ CUtensorMap tmS,
                const __grid_constant__ CUtensorMap tmdS, const __grid_constant__ CUtensorMap tmdq,
                const __grid_constant__ CUtensorMap tmdk, GradParams p) {
  extern __shared__ uint8_t smem_raw[];
  GradSmem& sm = *reinterpret_cast<GradSmem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, hh = warp >> 2;          // TMEM quadrant, column half
  const uint32_t lo = (uint32_t)(32 * q) << 16;
  const int i = 16 * q + (lane & 15);              // token of this thread
  const bool up = lane >= 16;                      // upper lanes: k's side, lower: q's
  const int T = p.d.T, N = chunks(T), grp = GROUP ? p.d.H / p.d.Hk : 1;
  const unsigned total = (unsigned)((size_t)p.d.B * p.d.Hk * N);
  const WaitCtx wc{&sm.abort, p.status, p.timeout_ns};
  uint32_t lfull = 0, lde = 0, lkq = 0;  // loads so far
  auto first_head = [&](unsigned id) {
    const int kh = id / N, b = kh / p.d.Hk;
    return b * p.d.H + (kh - b * p.d.Hk) * grp;
  };
  // Tiles of 64 columns of d_v: dY, S and dS and, with the first, the gates; and D and E, whose place
  // is free later. One copy for the first lane of a warp (issuing one takes about 100 cycles). A
  // copy may land before its barrier has been told.
  auto load_slice = [&](int bh, int n, int sl, GradGates* gates) {
    ++lfull;
    if (lane != 0) return;
    const int w = warp & 1;
    if (warp == 0) {
      mbar_arrive_expect_tx(&sm.full, 5 * TILE + (sl == 0 ? (uint32_t)sizeof(GradGates) : 0u));
      tma_load_3d(sm.O, &tmO, &sm.full, 64 * sl, n * C, bh);
    } else if (warp == 1) {
      if (sl == 0)
        bulk_load(gates,
                  reinterpret_cast<const char*>(p.gates) + ((size_t)bh * N + n) * sizeof(GateBlock) +
                      GradGates::offset,
                  sizeof(GradGates), &sm.full);
    } else if (warp >= 4 && warp < 6) {
      tma_load_3d(sm.S + w * TILE, &tmS, &sm.full, 64 * w, 64 * sl, bh * N + n);
    } else if (warp >= 6) {
      tma_load_3d(sm.dS + w * TILE, &tmdS, &sm.full, 64 * w, 64 * sl, bh * N + n);
    }
  };
  const int rows = dvp(p.d);
  auto load_de = [&](int bh, int n, int sl) {
    ++lde;
    if (lane != 0 || warp >= 4) return;
    const int w = warp & 1;
    if (warp == 0) mbar_arrive_expect_tx(&sm.de, 4 * TILE);
    tma_load_3d((warp < 2 ? sm.D : sm.E) + w * TILE, warp < 2 ? &tmD : &tmE, &sm.de, 0,
                w * rows + 64 * sl, bh * N + n);
  };
  // Tiles of Q (warps 4 and 5) and K (6 and 7)
  uint8_t* const kq_tile = (warp < 6 ? sm.Q : sm.K) + (warp & 1) * TILE;
  auto load_kq = [&](unsigned id) {
    const int kh = id / N, t0 = (id - kh * N) * C;
    ++lkq;
    if (warp < 4 || lane != 0) return;
    mbar_arrive_expect_tx(&sm.kq, TILE);
    tma_load_3d(kq_tile, warp < 6 ? &tmQ : &tmK, &sm.kq, 64 * (warp & 1), t0, kh);
  };
  if (tid == 0) {
    sm.abort = 0;
    mbar_init(&sm.kq, 4);
    mbar_init(&sm.full, 1);
    mbar_init(&sm.de, 1);
    mbar_init(&sm.mma, 1);
    fence_mbar_init();
  }
  const int nsl = (p.d.dv + 63) / 64;
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();
  load_slice(first_head(blockIdx.x), blockIdx.x % N, 0, &sm.gates[0]);
  load_de(first_head(blockIdx.x), blockIdx.x % N, 0);
  load_kq(blockIdx.x);
  __syncwarp();
  const uint32_t tb = sm.tmem_base;
  const uint32_t sQ = smem_u32(sm.Q), sK = smem_u32(sm.K), sX = smem_u32(sm.D), sY = smem_u32(sm.E);
  const uint32_t id_f = idesc_bf16(64, 64, false, true), id_h = idesc_bf16(64, 64, true, true);
  const uint32_t id_t = idesc_bf16(64, 128, false, true);
  const uint32_t id_m = idesc_bf16(64, 128, true, true);
  constexpr int XW = GROUP ? 8 : 16;  // columns of X and Yn at a time, as the registers allow
  uint32_t nfull = 0, nde = 0, nmma = 0, nkq = 0, nhead = 0;  // phases and heads so far

  bool stop = false;
  for (unsigned id = blockIdx.x; id < total; id += gridDim.x) {
  const int kh = id / N, n = id - kh * N, t0 = n * C, bh0 = first_head(id);
  F2 acc[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) acc[e] = f2(0.f, 0.f);

  for (int hv = 0; hv < grp; ++hv, ++nhead) {
    const int bh = bh0 + hv;
    const GradGates& g = sm.gates[nhead & 1];
    // The slice after the last one of this head, of the next head or (behind what follows here) the
    // next chunk; whether there is one
    auto next = [&](int& bh1, int& n1) -> bool {
      const unsigned id1 = id + (hv + 1 < grp ? 0u : gridDim.x);
      bh1 = hv + 1 < grp ? bh + 1 : first_head(id1);
      n1 = id1 % N;
      return id1 < total;
    };
    F2 ss = f2(0.f, 0.f);  // <dS, S>
    for (int sl = 0; sl < nsl; ++sl) {
      mbar_wait(&sm.full, nfull++ & 1, wc, W_G_FULL);
      mbar_wait(&sm.de, nde++ & 1, wc, W_G_DE);
      __syncwarp();
      if (tid == 0) {
        tc_fence_after();
        const uint32_t sO = smem_u32(sm.O), sD = smem_u32(sm.D), sE = smem_u32(sm.E);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t on = (sl > 0 || kk > 0) ? 1u : 0u;
          const uint64_t ao = desc_at(sw128_desc(sO, 16, 1024), kk * 32);
          const uint64_t ad = desc_at(sw128_desc(sD, TILE, 1024), kk * 2048);
          const uint64_t ae = desc_at(sw128_desc(sE, TILE, 1024), kk * 2048);
          const uint64_t adl = desc_at(ad, TILE), ael = desc_at(ae, TILE);  // the remainders
          const uint64_t bs = desc_at(sw128_desc(smem_u32(sm.S), TILE, 1024), kk * 2048);
          const uint64_t bd = desc_at(sw128_desc(smem_u32(sm.dS), TILE, 1024), kk * 2048);
          umma_bf16(tb + COL_B, ao, ad, id_f, on);                  // F
          umma_bf16(tb + COL_B, ao, adl, id_f, 1);
          umma_bf16(tb + COL_B + 64, ae, ad, id_h, on);             // H
          umma_bf16(tb + COL_B + 64, ae, adl, id_h, 1);
          umma_bf16(tb + COL_B + 64, ael, ad, id_h, 1);
          umma_bf16(tb + COL_A, ao, bs, id_t, on);                  // t
          umma_bf16(tb + COL_A + LANE16, ae, bs, id_m, on);         // u
          umma_bf16(tb + COL_A + LANE16, ael, bs, id_m, 1);
          umma_bf16(tb + COL_B + LANE16, ad, bd, id_m, on);         // z
          umma_bf16(tb + COL_B + LANE16, adl, bd, id_m, 1);
        }
        umma_commit(&sm.mma);
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t off = (uint32_t)(tid + 256 * k) * 16;
        const uint4 x = *reinterpret_cast<const uint4*>(sm.S + off);
        const uint4 y = *reinterpret_cast<const uint4*>(sm.dS + off);
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          ss = fma2(f2(bf16_lo(xw[e]), bf16_hi(xw[e])), f2(bf16_lo(yw[e]), bf16_hi(yw[e])), ss);
      }
      if (sl == 0 && warp == 2 && g.fac == 0.f) {
        const GatePair gp = chunk_gates(load_gates(p.beta, p.log_alpha, (size_t)bh * T, t0, T));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          sm.Lh[lane + 32 * k] = gp.Lh[k];
          sm.Ll[lane + 32 * k] = gp.Ll[k];
          sm.seg[lane + 32 * k] = gp.seg[k];
        }
      }
      mbar_wait(&sm.mma, nmma++ & 1, wc, W_G_MMA);
      // S and dS are read
      stop = __syncthreads_or(*reinterpret_cast<volatile int*>(&sm.abort));
      if (stop) break;
      // the next slice; X and Yn come before the next head's D and E
      if (sl + 1 < nsl) {
        load_slice(bh, n, sl + 1, nullptr);
        load_de(bh, n, sl + 1);
      } else {
        int bh1, n1;
        if (next(bh1, n1)) load_slice(bh1, n1, 0, &sm.gates[(nhead + 1) & 1]);
      }
      __syncwarp();
    }
    if (stop) break;
    float s0, s1;
    get2(ss, s0, s1);
    s0 += s1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
    if (lane == 0) sm.red[warp] = s0;
    tc_fence_after();
    // ---- X and Yn: lower lanes, columns [32 hh, 32 hh + 32)
    const float rx = p.scale * g.ra[i], ry = -g.be[i] * g.ra[i];
    float db = 0.f;
#pragma unroll
    for (int it = 0; it < 2 * 32 / XW; ++it) {
      const bool second = it >= 32 / XW;  // Yn after X, as the registers allow
      float f[XW];
      const int hf = it % (32 / XW), j0 = 32 * hh + XW * hf;
      tmem_ld(tb + COL_B + (second ? 64 : 0) + lo + j0, f);
      tmem_ld_wait();
      if (!up) {
        const int keep = i - j0 + (second ? 0 : 1);  // the first columns: left of the diagonal (X: and on it)
        const float r = second ? ry : rx;
        if (second) {
#pragma unroll
          for (int e = 0; e < XW; ++e) db = e == keep ? f[e] : db;
        }
        if (g.fac != 0.f) {
#pragma unroll
          for (int e = 0; e < XW; e += 4) {
            const float4 c = *reinterpret_cast<const float4*>(g.cb + j0 + e);
            const float cv[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) f[e + u] = e + u < keep ? f[e + u] * (r * cv[u]) : 0.f;
          }
        } else {  // a reset, or decays whose factors leave float32
          const float Lh = sm.Lh[i], Ll = sm.Ll[i];
          const int seg = sm.seg[i];
#pragma unroll
          for (int e = 0; e < XW; ++e) {
            const int j = j0 + e;
            const float m = g.cb[j] * expf(fminf((Lh - sm.Lh[j]) + (Ll - sm.Ll[j]), 0.f));
            f[e] = sm.seg[j] == seg && e < keep ? f[e] * (r * m) : 0.f;
          }
        }
#pragma unroll
        for (int cc = 0; cc < XW / 8; ++cc)
          put_split8((second ? sY : sX) + sw128_off(i, 4 * hh + XW / 8 * hf + cc), f + 8 * cc);
      }
      __syncwarp();
    }
    if (!up && (i >> 5) == hh && t0 + i < T) p.dbeta[(size_t)bh * T + t0 + i] = __float2bfloat16_rn(db);
    fence_proxy_async_smem();
    tc_fence_before();
    if (hv == 0) mbar_wait(&sm.kq, nkq++ & 1, wc, W_G_KQ);
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {  // xk over F and H
        const uint64_t ax = desc_at(sw128_desc(sX, 16, 1024), kk * 32);
        const uint64_t bk = desc_at(sw128_desc(sK, TILE, 1024), kk * 2048);
        umma_bf16(tb + COL_B, ax, bk, id_t, kk > 0);
        umma_bf16(tb + COL_B, desc_at(ax, TILE), bk, id_t, 1);
      }
    }
    __syncwarp();
    // ---- t (lower) and u (upper); z (upper)
    const uint8_t* mine = (up ? sm.K : sm.Q) + hh * TILE;
    const float ca = up ? g.bG[i] : g.q[i], cz = up ? g.bw[i] : 0.f;
    float xs, ps, zs;
    const F2 ca2 = f2(ca, ca), cz2 = f2(cz, cz);
    F2 dv = f2(0.f, 0.f), dz = dv;
    if (!GROUP) {
#pragma unroll
      for (int e = 0; e < 32; ++e) acc[e] = dv;
    }
#pragma unroll
    for (int cc = 0; cc < 8; ++cc) {
      float v[8], z[8], x[8];
      tmem_ld8(tb + COL_A + lo + 64 * hh + 8 * cc, v);
      tmem_ld8(tb + COL_B + lo + 64 * hh + 8 * cc, z);  // lower lanes: unused (xk in flight)
      row8(x, mine, i, cc);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const F2 ve = f2(v[e], v[e + 1]), ze = up ? f2(z[e], z[e + 1]) : f2(0.f, 0.f);
        const F2 xe = f2(x[e], x[e + 1]);
        F2& s = acc[4 * cc + e / 2];
        dv = fma2(ve, xe, dv);
        dz = fma2(ze, xe, dz);
        s = fma2(ca2, ve, fma2(cz2, ze, s));
      }
    }
    {
      float a, c;
      get2(dv, a, c);
      xs = ca * (a + c);
      get2(dz, a, c);
      zs = cz * (a + c);
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const uint64_t bq = desc_at(sw128_desc(sQ, TILE, 1024), kk * 2048);
        const uint64_t bk = desc_at(sw128_desc(sK, TILE, 1024), kk * 2048);
        const uint64_t xt = desc_at(sw128_desc(sX, TILE, 1024), kk * 2048);
        const uint64_t yt = desc_at(sw128_desc(sY, TILE, 1024), kk * 2048);
        const uint64_t ay = desc_at(sw128_desc(sY, 16, 1024), kk * 32);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          umma_bf16(tb + COL_B + LANE16, desc_at(xt, part * TILE), bq, id_m, kk + part > 0);
          umma_bf16(tb + COL_B + LANE16, desc_at(yt, part * TILE), bk, id_m, 1);
          umma_bf16(tb + COL_A + LANE16, desc_at(ay, part * TILE), bk, id_t, kk + part > 0);
        }
      }
      umma_commit(&sm.mma);
    }
    __syncwarp();
    mbar_wait(&sm.mma, nmma++ & 1, wc, W_G_MMA);
    __syncwarp();
    tc_fence_after();
    {
      int bh1, n1;
      if (next(bh1, n1)) load_de(bh1, n1, 0);  // X and Yn are read
    }
    __syncwarp();
    // ---- xk (lower) and ka (upper); yk (upper)
    dv = dz = f2(0.f, 0.f);
#pragma unroll
    for (int cc = 0; cc < 8; ++cc) {
      float v[8], z[8], x[8];
      tmem_ld8(tb + COL_B + lo + 64 * hh + 8 * cc, v);
      tmem_ld8(tb + COL_A + lo + 64 * hh + 8 * cc, z);  // lower lanes: t, used above
      row8(x, mine, i, cc);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const F2 ve = f2(v[e], v[e + 1]), ye = up ? f2(z[e], z[e + 1]) : f2(0.f, 0.f);
        const F2 xe = f2(x[e], x[e + 1]);
        F2& s = acc[4 * cc + e / 2];
        dv = fma2(ve, xe, dv);
        dz = fma2(ye, xe, dz);
        s = add2(s, add2(ve, ye));
      }
    }
    {  // q.xk, or k.(yk - ka)
      float a, c, y0, y1;
      get2(dv, a, c);
      get2(dz, y0, y1);
      ps = up ? (y0 + y1) - (a + c) : a + c;
    }
    xs += __shfl_xor_sync(0xffffffffu, xs, 16);
    ps += __shfl_xor_sync(0xffffffffu, ps, 16);
    zs += __shfl_xor_sync(0xffffffffu, zs, 16);
    if (!up) {
      sm.xs[hh][i] = xs;
      sm.ps[hh][i] = ps;
      sm.zs[hh][i] = zs;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {  // dlog_alpha: tokens 2 lane and 2 lane + 1
      const int j = 2 * lane;
      const float x0 = sm.xs[0][j] + sm.xs[1][j], x1 = sm.xs[0][j + 1] + sm.xs[1][j + 1];
      const float p0 = sm.ps[0][j] + sm.ps[1][j], p1 = sm.ps[0][j + 1] + sm.ps[1][j + 1];
      const float z0 = sm.zs[0][j] + sm.zs[1][j], z1 = sm.zs[0][j + 1] + sm.zs[1][j + 1];
      float sx = x0 + x1, sp = p0 + p1, sz = z0 + z1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float ux = __shfl_down_sync(0xffffffffu, sx, o), up_ = __shfl_down_sync(0xffffffffu, sp, o);
        const float uz = __shfl_up_sync(0xffffffffu, sz, o);
        if (lane + o < 32) {
          sx += ux;
          sp += up_;
        }
        if (lane >= o) sz += uz;
      }
      float gg = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) gg += sm.red[w];
      gg *= g.GC;
      const float before = __shfl_up_sync(0xffffffffu, sz, 1);
      const float z_lt = lane == 0 ? 0.f : before;
      // no pair reaches across the chunk's first token: its sum is zero, not what rounding left
      const float pair0 = lane == 0 ? 0.f : sp;
      const float after = __shfl_down_sync(0xffffffffu, sx + sp, 1);
      const float d0 = sx + pair0, d1 = (x1 + p1) + (lane == 31 ? 0.f : after);
      const size_t row = (size_t)bh * T + t0;
      const bool plain = g.fac != 0.f;  // no reset in the chunk
      const bool r0 = !plain && sm.seg[j] != (j > 0 ? sm.seg[j - 1] : 0);
      const bool r1 = !plain && sm.seg[j + 1] != sm.seg[j];
      if (t0 + j < T)
        p.dlog_alpha[row + j] = __float2bfloat16_rn(
            r0 ? 0.f : d0 + z_lt + gg);
      if (t0 + j + 1 < T)
        p.dlog_alpha[row + j + 1] = __float2bfloat16_rn(
            r1 ? 0.f : d1 + z_lt + z0 + gg);
    }
    __syncthreads();  // the next head overwrites the gates and the sums
  }
  if (stop) break;
  // ---- dq and dk over Q and K (every product has read them)
#pragma unroll
  for (int cc = 0; cc < 8; ++cc) {
    float a[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) get2(acc[4 * cc + e], a[2 * e], a[2 * e + 1]);
    st_shared_v4((up ? sK : sQ) + hh * TILE + sw128_off(i, cc), pack_bf16(a[0], a[1]),
                 pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]), pack_bf16(a[6], a[7]));
  }
  fence_proxy_async_smem();
  tc_fence_before();
  stop = __syncthreads_or(*reinterpret_cast<volatile int*>(&sm.abort));
  if (warp >= 4 && lane == 0) {  // a tile each, whose place the next chunk's takes
    if (64 * (warp & 1) < p.d.dk) {
      tma_store_3d(warp < 6 ? &tmdq : &tmdk, kq_tile, 64 * (warp & 1), t0, kh);
      tma_store_commit();
      tma_store_wait_read();
    }
  }
  if (stop) break;
  if (id + gridDim.x < total) load_kq(id + gridDim.x);
  __syncwarp();
  }
  if (tid == 0) {  // every load has landed
    mbar_drain(&sm.full, (lfull - 1) & 1, wc, W_G_DRAIN);
    mbar_drain(&sm.de, (lde - 1) & 1, wc, W_G_DRAIN);
    mbar_drain(&sm.kq, (lkq - 1) & 1, wc, W_G_DRAIN);
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tb, kCols);
  }
}

template <bool GROUP>
static cudaError_t launch(const CUtensorMap (&m)[9], const GradParams& p, unsigned work, cudaStream_t st) {
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!bit || !(set.load() & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(
        grad_kernel<GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit);
  }
  const unsigned most = 2 * 148;
  const cudaError_t e =
      launch_after(launches_early(p.d, false), grad_kernel<GROUP>, work < most ? work : most, kThreads, kSmem, st, m[0], m[1], m[2],
                   m[3], m[4], m[5], m[6], m[7], m[8], p);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_grad(const Args& a, cudaStream_t st) {
  using gradlev::tc::make_map_bf16_3d;
  const Dims& d = a.d;
  const uint64_t N = chunks(d.T), kh = (uint64_t)d.B * d.Hk, bh = d.BH();
  CUtensorMap m[9];
  if (!make_map_bf16_3d(&m[0], a.q, d.dk, d.T, kh, C) || !make_map_bf16_3d(&m[1], a.k, d.dk, d.T, kh, C) ||
      !make_map_bf16_3d(&m[2], a.dy, d.dv, d.T, bh, C) ||
      !make_map_bf16_3d(&m[3], a.sv.D, C, 2 * dvp(d), bh * N, 64) ||
      !make_map_bf16_3d(&m[4], a.E, C, 2 * dvp(d), bh * N, 64) ||
      !make_map_bf16_3d(&m[5], a.sv.S, 128, dvp(d), bh * N, 64) ||
      !make_map_bf16_3d(&m[6], a.dS, 128, dvp(d), bh * N, 64) ||
      !make_map_bf16_3d(&m[7], a.dq, d.dk, d.T, kh, C) ||
      !make_map_bf16_3d(&m[8], a.dk_, d.dk, d.T, kh, C))
    return cudaErrorInvalidValue;
  GradParams p{d, a.beta, a.log_alpha, a.sv.gates, a.scale, a.status, a.timeout_ns,
               static_cast<bf16*>(a.dbeta), static_cast<bf16*>(a.dlog_alpha)};
  return d.H > d.Hk ? launch<true>(m, p, (unsigned)(N * kh), st) : launch<false>(m, p, (unsigned)(N * kh), st);
}

}  // namespace tc
}  // namespace delta
}  // namespace gradlev
