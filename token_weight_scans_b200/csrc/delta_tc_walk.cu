// Tensor-core gated delta rule: the state recurrence over the chunks of one scan, one CTA
// per (b, h, 128 rows of d_v). Matrices of struct Mats in delta_tc.h; everything on the
// state is transposed (rows of d_v in the 128 TMEM lanes, tokens or d_k in the columns),
// so that the two operands made from the previous product stay in tensor memory:
//
//   forward                                backward (chunks in reverse, S is dS)
//   D^T  = V^T T0^T + S W^T                E^T = dY^T PT + S Wb^T
//   S    = G_C S + (beta w D)^T K          S   = G_C S + dY^T (scale G Q) + E^T (-beta G K)
//   Y^T  = S (scale G Q)^T + D^T Pb^T      dV  = beta E
//
// The chain through a chunk is: S to bf16 (TMEM -> registers -> TMEM), the product with W,
// its result to bf16, the product with K. All else runs beside it: V^T T0^T of the next
// chunk and the outputs' products are issued into the gaps of the chain, and their results
// leave through an output warpgroup. Without SPLIT one product of N = 128 takes S through W
// and Q together.
//
// SPLIT (a forward whose last state is asked for): every operand of the state that is not
// exact in bf16 comes as a sum of two bf16 (S, W, T0, beta w D), three products in place of
// one, so that S carries 16 bits through the chunks and the float32 state it ends with is
// good to 1e-5. Training needs no such state and takes single products.
//
// Warp roles (16): 0 and 3 TMA producers, 1 MMA issuer (owns TMEM), 2 copies the gates in,
// 4-11 two chain warpgroups (each half of the columns), which also leave S and D^T (E^T) for
// the kernels after, 12-15 scaling of Q by scale G, and Y (dV): 16-lane TMEM loads in the
// layout of 8 x 8 fragments, transposed on the way to shared memory (stmatrix) so that tokens
// become rows, and TMA stores. D^T and E^T stay as they are, a chunk's tokens contiguous.
//
// Measured (B8 H16 T4096 d 128, 128 CTAs of 64 chunks): forward 190 us, backward 180 us, of
// 2304 and 2176 bytes per token: 6.3 TB/s, the measured copy bandwidth (6.47). Where HBM does
// not bound it, a chunk takes 2.3 us (forward), 2.9 us with SPLIT: the chain, two products and
// two passes of the state or D through registers.
//
// Each chunk's tiles come in three groups with a two-deep ring of their own, since they are
// done with at different times: V (dY) with T0 (PT), W with Q, K with Pb.
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

constexpr int NS = 2;             // TMA stages
constexpr int GS = 3;             // gate slots
constexpr int kThreads = 512;

// TMEM columns
constexpr uint32_t COL_S = 0;      // float32 state, 128
constexpr uint32_t COL_SH = 128;   // bf16 state, 64
constexpr uint32_t COL_DB = 192;   // bf16 D (E), 32
constexpr uint32_t COL_U = 224;    // bf16 beta w D, 32
constexpr uint32_t COL_D = 256;    // D^T (E^T) accumulator, 64, and Y^T, 64; two such pairs
// SPLIT has one set: D^T in two parts that the chain adds (the products with T0 and W, and with
// their remainders), then Y^T: the three take one product of N = 192
constexpr uint32_t COL_YS = 384;   // SPLIT: Y^T
constexpr uint32_t COL_SL = 448;   // SPLIT: remainder of the state, 64; once the products with W
constexpr uint32_t COL_UL = 448;   // have read it, that of beta w D, 32

// A chunk's gates: the piece of GateBlock that the direction needs, as it lies there.
template <bool BWD> struct GateSlot;
template <> struct GateSlot<false> {
  float u[C], GC, pad[3], q[C];         // bw .. q
  static constexpr int offset = 0;
};
template <> struct GateSlot<true> {
  float GC, pad[3], q[C], u[C], be[C];  // GC .. be
  static constexpr int offset = C * sizeof(float);
};
static_assert(sizeof(GateSlot<false>) % 16 == 0 && sizeof(GateSlot<true>) % 16 == 0 &&
              sizeof(GateBlock) % 16 == 0, "bulk copies");

template <bool BWD>
struct Bars {
  GateSlot<BWD> gates[GS];
  uint64_t full[3][NS], empty[3][NS];   // per group of tiles
  uint64_t scaled[NS];
  uint64_t gfull[GS], gempty[GS];
  uint64_t sready[2];                   // (SPLIT: in two halves of each warp's columns)
  uint64_t sscaled, dfull, uready, sfull, done;
  uint64_t yfull[2], yfree[2];          // per accumulator pair
  uint32_t tmem_base;
  int abort;
};
enum { VT = 0, WQ = 1, KP = 2 };

// The rings. VT: V (dY), T0 (PT), SPLIT also the remainder of T0. WQ: per 64 columns of d_k the
// W (Wb) tile, SPLIT the remainder of W, and the Q tile next to each other (128 or 192 rows of
// one operand). KP: K, forward also Pb.
template <bool BWD, bool SPLIT>
struct Layout {
  static constexpr int v = 0, t = 2 * TILE, tl = 3 * TILE;
  static constexpr int w = 0, wl = TILE, q = SPLIT ? 2 * TILE : TILE;
  static constexpr int wq = q + TILE;    // from one k-block to the next
  static constexpr int k = 0, p = 2 * TILE;
  static constexpr int vt_bytes = SPLIT ? 4 * TILE : 3 * TILE;
  static constexpr int wq_bytes = SPLIT ? 6 * TILE : 4 * TILE;
  static constexpr int kp_bytes = BWD ? 2 * TILE : 3 * TILE;
  static constexpr int wq0 = NS * vt_bytes, kp0 = wq0 + NS * wq_bytes;
  static constexpr bool staged = !SPLIT;   // S and D^T through shared memory and TMA
  static constexpr int stage_s = kp0 + NS * kp_bytes, stage_o = stage_s + (staged ? 2 * BIG : 0);
  static constexpr int stage_d = stage_o + 2 * TILE;
  static constexpr int bars = stage_d + (staged ? 2 * TILE : 0);  // (SPLIT: Y alone is staged)
  static constexpr size_t smem = bars + sizeof(Bars<BWD>) + 1024;
  static_assert(smem <= 227 * 1024, "over the shared memory of a CTA");
  static constexpr int vt(int s) { return s * vt_bytes; }
  static constexpr int wq_at(int s) { return wq0 + s * wq_bytes; }
  static constexpr int kp(int s) { return kp0 + s * kp_bytes; }
};

enum : uint32_t {
  W_TMA = 0x901, W_TMA_DRAIN, W_FULL = 0x911, W_SCALED, W_SREADY, W_UREADY, W_YFREE, W_DONE,
  W_GATE = 0x921, W_C_SFULL = 0x931, W_C_DFULL, W_C_GATE, W_O_FULL = 0x941, W_O_GATE, W_O_Y,
};

struct WalkParams {
  Dims d;
  const float* gates;
  DeviceStatus* status;
  uint64_t timeout_ns;
  const float* S0;       // forward start
  const float* log_alpha;
  const bf16* dST;       // backward start
  float* ST;             // forward end
  bf16* dS0;             // backward end
  bf16* y;               // forward
  bf16* D;               // forward: D^T, backward: E^T (null: not kept)
  bf16* states;          // chunk-start (chunk-end) states, or null
  // Segments (delta_tc_seg.cu): CTA u < nsl B H segs walks segment seg0 + u / (nsl B H); the
  // slice past the last one carries the identity. CTAs past those carry it through the last
  // segment.
  int nseg, seg_chunks, seg0, segs, nsl;
  int inject;            // test hook
  int sum;               // states alone: nothing is left for other kernels but loc and M
  const float* init;     // [B*H][nseg][dvp][128] states the segments start from, or null
  float *loc, *M;        // [B*H][nseg][dvp][128], [B*H][nseg][128][128]
};

__device__ __forceinline__ void st_tmem32(uint32_t col, const uint32_t (&r)[32]) {
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
  tmem_st32(col, v);
}
__device__ __forceinline__ void st_tmem16(uint32_t col, const uint32_t (&r)[16]) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
  tmem_st16(col, v);
}
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t hi) {
  return pack_bf16(a - bf16_lo(hi), b - bf16_hi(hi));
}

// Barrier `id` among `nthreads` threads; whether any of them brought `pred`.
__device__ __forceinline__ bool named_bar_or(uint32_t id, uint32_t nthreads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}

// x *= factor[row] on a [64 tokens x 128] tile in place (its k-blocks `step` bytes apart), by
// 128 threads; the loads go out together.
__device__ __forceinline__ void scale_tile(uint32_t tile, uint32_t step, const float* factor, int t) {
  uint4 v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = ld_shared_v4(tile + (k >> 2) * step + (t + 128 * (k & 3)) * 16);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t in = (uint32_t)(t + 128 * (k & 3)) * 16;
    const float f = factor[in >> 7];
    st_shared_v4(tile + (k >> 2) * step + in, pack_bf16(f * bf16_lo(v[k].x), f * bf16_hi(v[k].x)),
                 pack_bf16(f * bf16_lo(v[k].y), f * bf16_hi(v[k].y)),
                 pack_bf16(f * bf16_lo(v[k].z), f * bf16_hi(v[k].z)),
                 pack_bf16(f * bf16_lo(v[k].w), f * bf16_hi(v[k].w)));
  }
}

// 64 float32 columns of 16 TMEM lanes as 8 x 8 fragments: registers 4 g .. 4 g + 3 hold, of
// columns 8 g + 2 (lane % 4) and the one after, rows lane / 4 (first two) and lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_frag64(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void stmatrix_trans4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                                uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// 16 state rows (fragments of 64 tokens) into the [64 tokens x 128] tile, tokens as rows; the
// rows start at `row` (a multiple of 16).
__device__ __forceinline__ void put_frag64(uint32_t tile, int row, const float (&v)[32]) {
  const int lane = threadIdx.x & 31, m = lane >> 3;
  const uint32_t block = tile + (row >> 6) * TILE;
  const uint32_t c = ((row & 63) >> 3) + (m & 1);
#pragma unroll
  for (int g = 0; g < 8; g += 2)
    stmatrix_trans4(block + sw128_off(8 * (g + (m >> 1)) + (lane & 7), c),
                    pack_bf16(v[4 * g], v[4 * g + 1]), pack_bf16(v[4 * g + 2], v[4 * g + 3]),
                    pack_bf16(v[4 * g + 4], v[4 * g + 5]), pack_bf16(v[4 * g + 6], v[4 * g + 7]));
}

}  // namespace

template <bool BWD, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    walk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmW,
                const __grid_constant__ CUtensorMap tmWl, const __grid_constant__ CUtensorMap tmT,
                const __grid_constant__ CUtensorMap tmTl, const __grid_constant__ CUtensorMap tmP,
                const __grid_constant__ CUtensorMap tmS, const __grid_constant__ CUtensorMap tmY,
                const __grid_constant__ CUtensorMap tmD, WalkParams p) {
  using L = Layout<BWD, SPLIT>;
  constexpr int NY = SPLIT ? 1 : 2;   // accumulator pairs
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Bars<BWD>& sm = *reinterpret_cast<Bars<BWD>*>(base + L::bars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int BH = p.d.B * p.d.H, per_seg = p.nsl * BH;
  const bool extra = (int)blockIdx.x >= per_seg * p.segs;
  const int in_seg = extra ? blockIdx.x - per_seg * p.segs : blockIdx.x % per_seg;
  const int seg = extra ? p.nseg - 1 : p.seg0 + blockIdx.x / per_seg;
  const int bh = extra ? in_seg : in_seg / p.nsl, slice = extra ? 0 : in_seg - bh * p.nsl;
  const bool ident = extra || slice == dvp(p.d) >> 7;  // carries the identity: the segment's map
  const int n0 = ident ? 0 : slice * 128;
  const bool carry = p.sum || ident;                 // the end state is all that is wanted
  const bool outputs = !BWD && !carry;               // the forward's products for Y
  const size_t sg = (size_t)bh * p.nseg + seg;
  const int b = bh / p.d.H, h = bh - b * p.d.H;
  const int kh = b * p.d.Hk + h / (p.d.H / p.d.Hk);
  const int T = p.d.T, N = chunks(T);
  const int c0 = seg * p.seg_chunks, NC = min(N - c0, p.seg_chunks);  // the chunks walked
  auto cg = [&](int c) { return BWD ? c0 + NC - 1 - c : c0 + c; };
  const WaitCtx wc{&sm.abort, p.status, p.timeout_ns};

  if (threadIdx.x == 0) {
    sm.abort = 0;
    for (int s = 0; s < NS; ++s) {
      for (int r = 0; r < 3; ++r) {
        mbar_init(&sm.full[r][s], 1);
        mbar_init(&sm.empty[r][s], 1);
      }
      mbar_init(&sm.scaled[s], 4);
    }
    for (int g = 0; g < GS; ++g) {
      mbar_init(&sm.gfull[g], 1);
      mbar_init(&sm.gempty[g], 12);  // the chain's 8 warps, 4 that scale Q
    }
    mbar_init(&sm.sready[0], 8);
    mbar_init(&sm.sready[1], 8);
    mbar_init(&sm.sscaled, 8);
    mbar_init(&sm.dfull, 1);
    mbar_init(&sm.uready, 8);
    mbar_init(&sm.sfull, 1);
    mbar_init(&sm.done, 1);
    for (int y = 0; y < 2; ++y) {
      mbar_init(&sm.yfull[y], 1);
      mbar_init(&sm.yfree[y], 4);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();  // nothing before this line reads or writes global memory
  grid_dep_launch();
  const uint32_t tb = sm.tmem_base;

  if (warp == 0 || warp == 3) {
    // ------------------------------------------------------------ TMA producers
    // warp 0: V with T0, and K with Pb; warp 3: W with Q
    if (lane == 0) {
      int issued[3] = {0, 0, 0};
      auto open = [&](int r, int c, int bytes) -> bool {
        if (!mbar_wait(&sm.empty[r][c % NS], ((c / NS) & 1) ^ 1, wc, W_TMA)) return false;
        mbar_arrive_expect_tx(&sm.full[r][c % NS], bytes);
        issued[r] = c + 1;
        return true;
      };
      for (int c = 0; c < NC; ++c) {
        const int s = c % NS, t0 = cg(c) * C;
        if (warp == 0) {
          uint8_t* a = base + L::vt(s);
          uint64_t* f = &sm.full[VT][s];
          if (!open(VT, c, L::vt_bytes)) break;
          const int tv = ident ? N * C : t0;  // past the last token: zeros
          tma_load_3d(a + L::v, &tmV, f, n0, tv, bh);
          tma_load_3d(a + L::v + TILE, &tmV, f, n0 + 64, tv, bh);
          tma_load_3d(a + L::t, &tmT, f, 0, t0, bh);
          if (SPLIT) tma_load_3d(a + L::tl, &tmTl, f, 0, t0, bh);
          a = base + L::kp(s);
          f = &sm.full[KP][s];
          if (!open(KP, c, L::kp_bytes - (!BWD && carry ? TILE : 0))) break;
          tma_load_3d(a + L::k, &tmK, f, 0, t0, kh);
          tma_load_3d(a + L::k + TILE, &tmK, f, 64, t0, kh);
          if (outputs) tma_load_3d(a + L::p, &tmP, f, 0, t0, bh);
        } else {
          uint8_t* a = base + L::wq_at(s);
          uint64_t* f = &sm.full[WQ][s];
          if (!open(WQ, c, L::wq_bytes - (!BWD && carry ? 2 * TILE : 0))) break;
          for (int kb = 0; kb < 2; ++kb) {
            if (BWD || outputs) tma_load_3d(a + L::q + kb * L::wq, &tmQ, f, 64 * kb, t0, kh);
            tma_load_3d(a + L::w + kb * L::wq, &tmW, f, 64 * kb, t0, bh);
            if (SPLIT) tma_load_3d(a + L::wl + kb * L::wq, &tmWl, f, 64 * kb, t0, bh);
          }
        }
      }
      // teardown: every load issued has landed
      for (int r = 0; r < 3; ++r)
        for (int c = issued[r] > NS ? issued[r] - NS : 0; c < issued[r]; ++c)
          mbar_drain(&sm.full[r][c % NS], (c / NS) & 1, wc, W_TMA_DRAIN);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t id_v = idesc_bf16(128, SPLIT ? 128 : 64, true, BWD);  // V^T T0^T, dY^T PT
      const uint32_t id_w = idesc_bf16(128, 64, false, false);    // S W^T, S Q^T, D^T Pb^T
      const uint32_t id_wq = idesc_bf16(128, 128, false, false);  // S [W; Q]^T, S [W; Wlo]^T
      const uint32_t id_wwq = idesc_bf16(128, 192, false, false); // S [W; Wlo; Q]^T
      const uint32_t id_u = idesc_bf16(128, 128, false, true);    // U^T K, E^T K
      const uint32_t id_o = idesc_bf16(128, 128, true, true);     // dY^T Q
      // D^T of chunk c = V^T T0^T. Its pair of accumulators is free once the chain has read D
      // (uready, waited by then) and the outputs have been taken.
      auto first = [&](int c) -> bool {
        const int s = c % NS;
        const uint32_t st = smem_u32(base + L::vt(s)), d = tb + COL_D + 128 * (c % NY);
        if (!mbar_wait(&sm.full[VT][s], (c / NS) & 1, wc, W_FULL)) return false;
        if (!SPLIT && !mbar_wait(&sm.yfree[c % NY], ((c / NY) & 1) ^ 1, wc, W_YFREE)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t av = desc_at(sw128_desc(st + L::v, TILE, 1024), kk * 2048);
          const uint32_t off = BWD ? kk * 2048 : kk * 32;
          umma_bf16(d, av, desc_at(sw128_desc(st + L::t, BWD ? TILE : 16, 1024), off), id_v, kk > 0);
        }
        if (!BWD) umma_commit(&sm.empty[VT][s]);
        return true;
      };
      bool ok = first(0);
      for (int c = 0; c < NC && ok; ++c) {
        const int s = c % NS, yb = c % NY;
        const uint32_t st = smem_u32(base + L::wq_at(s)), sv = smem_u32(base + L::vt(s));
        const uint32_t sk = smem_u32(base + L::kp(s));
        const uint32_t d = tb + COL_D + 128 * yb, y = SPLIT ? tb + COL_YS : d + 64;
        if (!mbar_wait(carry && !BWD ? &sm.full[WQ][s] : &sm.scaled[s], (c / NS) & 1, wc, W_SCALED)) break;
        if (!mbar_wait(&sm.sready[0], c & 1, wc, W_SREADY)) break;
        tc_fence_after();
        // D^T += S W^T, and without SPLIT Y^T = S Q^T in the same products
        if (!SPLIT && outputs) {
          umma_bf16_tmem_a(d, tb + COL_SH, sw128_desc(st + L::w, 16, 1024), id_w, 1);
          umma_bf16_tmem_a(y, tb + COL_SH, sw128_desc(st + L::q, 16, 1024), id_w, 0);
#pragma unroll
          for (int kk = 1; kk < 8; ++kk)
            umma_bf16_tmem_a(d, tb + COL_SH + 8 * kk,
                             desc_at(sw128_desc(st + L::w, 16, 1024), (kk >> 2) * L::wq + (kk & 3) * 32),
                             id_wq, 1);
        } else if (!SPLIT) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16_tmem_a(d, tb + COL_SH + 8 * kk,
                             desc_at(sw128_desc(st + L::w, 16, 1024), (kk >> 2) * L::wq + (kk & 3) * 32),
                             id_w, 1);
        } else {
          // the K steps in the order in which the two warpgroups convert S, so that the products
          // of the first half run while the second is converted
          bool got = !outputs || mbar_wait(&sm.yfree[0], (c & 1) ^ 1, wc, W_YFREE);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (half == 1) got = got && mbar_wait(&sm.sready[1], c & 1, wc, W_SREADY);
            if (!got) break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int kk = 4 * (j >> 1) + 2 * half + (j & 1);
              const uint32_t off = (kk >> 2) * L::wq + (kk & 3) * 32;
              const uint64_t bw = desc_at(sw128_desc(st + L::w, 16, 1024), off);
              if (outputs && kk > 0) {
                umma_bf16_tmem_a(d, tb + COL_SH + 8 * kk, bw, id_wwq, 1);
              } else {
                umma_bf16_tmem_a(d, tb + COL_SH + 8 * kk, bw, id_wq, 1);
                if (outputs)
                  umma_bf16_tmem_a(y, tb + COL_SH, desc_at(sw128_desc(st + L::q, 16, 1024), off), id_w, 0);
              }
              umma_bf16_tmem_a(d, tb + COL_SL + 8 * kk, bw, id_w, 1);
            }
          }
          if (!got) break;
        }
        if (!(p.inject && c == 1)) umma_commit(&sm.dfull);
        if (BWD) {
          umma_commit(&sm.yfull[yb]);
          if (!mbar_wait(&sm.sscaled, c & 1, wc, W_SREADY)) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // S += dY^T (scale G Q)
            umma_bf16(tb + COL_S, desc_at(sw128_desc(sv + L::v, TILE, 1024), kk * 2048),
                      desc_at(sw128_desc(st + L::q, L::wq, 1024), kk * 2048), id_o, 1);
          umma_commit(&sm.empty[VT][s]);
          umma_commit(&sm.empty[WQ][s]);
        } else {
          umma_commit(&sm.empty[WQ][s]);
          if (!SPLIT && c + 1 < NC && !first(c + 1)) break;
        }
        if (!mbar_wait(&sm.full[KP][s], (c / NS) & 1, wc, W_FULL)) break;
        if (!mbar_wait(&sm.uready, c & 1, wc, W_UREADY)) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {  // S += U^T K
          const uint64_t bk = desc_at(sw128_desc(sk + L::k, TILE, 1024), kk * 2048);
          umma_bf16_tmem_a(tb + COL_S, tb + COL_U + 8 * kk, bk, id_u, 1);
          if (SPLIT) umma_bf16_tmem_a(tb + COL_S, tb + COL_UL + 8 * kk, bk, id_u, 1);
        }
        umma_commit(&sm.sfull);
        if (!BWD) {
          if (outputs) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // Y^T += D^T Pb^T
              umma_bf16_tmem_a(y, tb + COL_DB + 8 * kk,
                               desc_at(sw128_desc(sk + L::p, 16, 1024), kk * 32), id_w, 1);
          }
          umma_commit(&sm.yfull[yb]);
        }
        umma_commit(&sm.empty[KP][s]);
        if ((BWD || SPLIT) && c + 1 < NC) ok = first(c + 1);
      }
      umma_commit(&sm.done);
      mbar_drain(&sm.done, 0, wc, W_DONE);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ gates
    if (lane == 0) {
      const char* src = reinterpret_cast<const char*>(p.gates) + GateSlot<BWD>::offset;
      int issued = 0;
      for (int c = 0; c < NC; ++c) {
        const int g = c % GS;
        if (!mbar_wait(&sm.gempty[g], ((c / GS) & 1) ^ 1, wc, W_GATE)) break;
        mbar_arrive_expect_tx(&sm.gfull[g], sizeof(GateSlot<BWD>));
        bulk_load(&sm.gates[g], src + ((size_t)bh * N + cg(c)) * sizeof(GateBlock),
                  sizeof(GateSlot<BWD>), &sm.gfull[g]);
        issued = c + 1;
      }
      for (int c = issued > GS ? issued - GS : 0; c < issued; ++c)
        mbar_drain(&sm.gfull[c % GS], (c / GS) & 1, wc, W_TMA_DRAIN);
    }
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ the chain
    const int q = warp & 3, hh = (warp - 4) >> 2;
    const uint32_t lo = (uint32_t)(32 * q) << 16;
    const int r = 32 * q + lane;           // row of the slice
    // rows and columns of the caller's states (S0, ST, dST, dS0 have no padding)
    const bool rok = n0 + r < p.d.dv;
    const size_t row = ((size_t)bh * p.d.dv + n0 + r) * p.d.dk;
    auto cok = [&](int col) { return rok && col < p.d.dk; };
    const int rows = dvp(p.d);
    // start state; S0 may hold anything where the first token is a reset
    const bool use_S0 = !BWD && p.S0 && !(p.log_alpha[(size_t)bh * p.d.T] < kResetLog);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      float v[32];
      const int col = 64 * hh + 32 * hf;
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = ident && col + e == r ? 1.f : 0.f;
      const float* from = p.init ? p.init + (sg * rows + n0 + r) * 128 : use_S0 ? p.S0 + row : nullptr;
      if (!carry && from) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (!p.init && !cok(col + 4 * e)) continue;
          const float4 u = *reinterpret_cast<const float4*>(from + col + 4 * e);
          v[4 * e] = u.x;
          v[4 * e + 1] = u.y;
          v[4 * e + 2] = u.z;
          v[4 * e + 3] = u.w;
        }
      }
      if (BWD && !carry && !p.init && p.dST) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!cok(col + 8 * e)) continue;
          const uint4 u = *reinterpret_cast<const uint4*>(p.dST + row + col + 8 * e);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            v[8 * e + 2 * f] = bf16_lo(w[f]);
            v[8 * e + 2 * f + 1] = bf16_hi(w[f]);
          }
        }
      }
      __syncwarp();
      tmem_st32(tb + COL_S + lo + col, v);
    }
    tmem_st_wait();
    bool ok = true;
    for (int c = 0; c < NC && ok; ++c) {
      const int g = c % GS, n = cg(c);
      const GateSlot<BWD>& gs = sm.gates[g];
      ok = mbar_wait_warp(&sm.gfull[g], (c / GS) & 1, wc, W_C_GATE);
      // every product of chunk c - 1 that reads the bf16 state was issued before this commit
      ok = ok && (c == 0 || mbar_wait_warp(&sm.sfull, (c - 1) & 1, wc, W_C_SFULL));
      if (!ok) break;
      tc_fence_after();
      const float GC = gs.GC;
      uint32_t pk[32];
      const uint32_t at = tb + COL_S + lo + 64 * hh;
      if constexpr (SPLIT) {  // 32 columns at a time (registers), each half as it is ready
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float v[32];
          tmem_ld32(at + 32 * hf, v);
          tmem_ld_wait();
          uint32_t hi[16], rest[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            hi[e] = pk[16 * hf + e] = pack_bf16(v[2 * e], v[2 * e + 1]);
            rest[e] = pack_rest(v[2 * e], v[2 * e + 1], hi[e]);
          }
          st_tmem16(tb + COL_SH + lo + 32 * hh + 16 * hf, hi);
          st_tmem16(tb + COL_SL + lo + 32 * hh + 16 * hf, rest);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.sready[hf]);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {  // the decay, read again: not before the update
          float v[32];
          tmem_ld32(at + 32 * hf, v);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] *= GC;
          tmem_st32(at + 32 * hf, v);
        }
      } else {
        // the bf16 copy first; the decayed state is only needed by the update (backward: by
        // dY^T Q)
        float v0[32], v1[32];
        tmem_ld32(at, v0);
        tmem_ld32(at + 32, v1);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          pk[e] = pack_bf16(v0[2 * e], v0[2 * e + 1]);
          pk[16 + e] = pack_bf16(v1[2 * e], v1[2 * e + 1]);
        }
        st_tmem32(tb + COL_SH + lo + 32 * hh, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.sready[0]);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          v0[e] *= GC;
          v1[e] *= GC;
        }
        tmem_st32(at, v0);
        tmem_st32(at + 32, v1);
        if (BWD) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.sscaled);
        }
      }
      if (p.states && !carry) {
        if (L::staged) {
          if (lane == 0) tma_store_wait_read_n<0>();  // the store of the chunk before
          __syncwarp();
          const uint32_t tile = smem_u32(base + L::stage_s + hh * BIG);
#pragma unroll
          for (int cc = 0; cc < 8; ++cc)
            st_shared_v4(tile + sw128_off(r, cc), pk[4 * cc], pk[4 * cc + 1], pk[4 * cc + 2],
                         pk[4 * cc + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tmS, base + L::stage_s + hh * BIG + 32 * q * 128, 64 * hh, n0 + 32 * q,
                         bh * N + n);
            tma_store_commit();
          }
        } else {
          uint4* out = reinterpret_cast<uint4*>(
              p.states + (((size_t)bh * N + n) * rows + n0 + r) * 128 + 64 * hh);
#pragma unroll
          for (int cc = 0; cc < 8; ++cc)
            out[cc] = make_uint4(pk[4 * cc], pk[4 * cc + 1], pk[4 * cc + 2], pk[4 * cc + 3]);
        }
      }
      // this warp's 32 factors, before the wait: shared memory is busy with operands after it
      float uf[32];
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 f = *reinterpret_cast<const float4*>(gs.u + 32 * hh + e);
        uf[e] = f.x;
        uf[e + 1] = f.y;
        uf[e + 2] = f.z;
        uf[e + 3] = f.w;
      }
      ok = mbar_wait_warp(&sm.dfull, c & 1, wc, W_C_DFULL);
      if (!ok) break;
      tc_fence_after();
      float v[32];
      tmem_ld32(tb + COL_D + 128 * (c % NY) + lo + 32 * hh, v);
      if constexpr (SPLIT) {
        float w[32];
        tmem_ld32(tb + COL_D + 64 + lo + 32 * hh, w);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] += w[e];
      } else {
        tmem_ld_wait();
      }
      uint32_t db[16];  // D (E) in bf16: 32 tokens of this row
      {
        uint32_t ub[16], rest[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float u0 = v[2 * e] * uf[2 * e], u1 = v[2 * e + 1] * uf[2 * e + 1];
          ub[e] = pack_bf16(u0, u1);
          db[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
          if (SPLIT) rest[e] = pack_rest(u0, u1, ub[e]);
        }
        st_tmem16(tb + COL_U + lo + 16 * hh, ub);
        if (!BWD) st_tmem16(tb + COL_DB + lo + 16 * hh, db);
        if (SPLIT) st_tmem16(tb + COL_UL + lo + 16 * hh, rest);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.uready);
      if (p.D && !carry) {
        if (L::staged) {  // a warp stores its own 32 rows x 32 tokens (64-byte rows and swizzle)
          if (lane == 0) tma_store_wait_read_n<1>();  // all but S of this chunk
          __syncwarp();
          uint8_t* const part = base + L::stage_d + (warp - 4) * 2048;
          const uint32_t at = smem_u32(part) + lane * 64;
#pragma unroll
          for (int cc = 0; cc < 4; ++cc)
            st_shared_v4(at + ((cc ^ ((lane >> 1) & 3)) << 4), db[4 * cc], db[4 * cc + 1],
                         db[4 * cc + 2], db[4 * cc + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tmD, part, 32 * hh, n0 + 32 * q, bh * N + n);
            tma_store_commit();
          }
        } else {
          uint4* out = reinterpret_cast<uint4*>(
              p.D + (((size_t)bh * N + n) * rows + n0 + r) * C + 32 * hh);
#pragma unroll
          for (int cc = 0; cc < 4; ++cc)
            out[cc] = make_uint4(db[4 * cc], db[4 * cc + 1], db[4 * cc + 2], db[4 * cc + 3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.gempty[g]);
    }
    if (lane == 0 && L::staged) tma_store_wait_all();
    float* inner = ident ? p.M + (sg * 128 + r) * 128 : carry ? p.loc + (sg * rows + n0 + r) * 128 : nullptr;
    float* end = !BWD && !carry && seg == p.nseg - 1 ? p.ST : nullptr;
    bf16* end16 = BWD && !carry && seg == 0 ? p.dS0 : nullptr;
    if (ok && (inner || end || end16) && mbar_wait_warp(&sm.sfull, (NC - 1) & 1, wc, W_C_SFULL)) {
      tc_fence_after();
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float v[32];
        const int col = 64 * hh + 32 * hf;
        tmem_ld32(tb + COL_S + lo + col, v);
        tmem_ld_wait();
        if (end16) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (cok(col + 8 * e))
              *reinterpret_cast<uint4*>(end16 + row + col + 8 * e) =
                  make_uint4(pack_bf16(v[8 * e], v[8 * e + 1]), pack_bf16(v[8 * e + 2], v[8 * e + 3]),
                             pack_bf16(v[8 * e + 4], v[8 * e + 5]), pack_bf16(v[8 * e + 6], v[8 * e + 7]));
        } else {
          float* o = inner ? inner + col : end + row + col;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (inner || cok(col + 4 * e))
              *reinterpret_cast<float4*>(o + 4 * e) =
                  make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
        __syncwarp();
      }
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------ scaled Q; outputs
    const int q = warp & 3, t = threadIdx.x & 127;
    const uint32_t lo = (uint32_t)(32 * q) << 16;
    auto scale_chunk = [&](int c) -> bool {
      const int s = c % NS, g = c % GS;
      if (!BWD && carry) return true;
      if (!mbar_wait_warp(&sm.full[WQ][s], (c / NS) & 1, wc, W_O_FULL)) return false;
      if (!mbar_wait_warp(&sm.gfull[g], (c / GS) & 1, wc, W_O_GATE)) return false;
      scale_tile(smem_u32(base + L::wq_at(s)) + L::q, L::wq, sm.gates[g].q, t);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.scaled[s]);
      return true;
    };
    // 128 rows x 64 tokens at TMEM column `col` to a [64 tokens x 128] tile of `map`, times
    // factor[token] if given
    uint8_t* const stage = base + L::stage_o;
    const uint32_t tile = smem_u32(stage);
    auto emit = [&](uint32_t col, const CUtensorMap* map, const float* factor, int t0, uint64_t* after) {
      if (t == 0) tma_store_wait_read_n<0>();  // the tile's last store
      named_bar_sync(1, 128);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float v[32];
        tmem_ld_frag64(tb + col + lo + hf * LANE16, v);
        tmem_ld_wait();
        if (after && hf == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(after);
        }
        if (factor) {
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const float2 f = *reinterpret_cast<const float2*>(factor + 8 * g + 2 * (lane & 3));
            v[4 * g] *= f.x;
            v[4 * g + 1] *= f.y;
            v[4 * g + 2] *= f.x;
            v[4 * g + 3] *= f.y;
          }
        }
        put_frag64(tile, 32 * q + 16 * hf, v);
      }
      fence_proxy_async_smem();
      named_bar_sync(1, 128);
      if (t == 0) {
        tma_store_3d(map, stage, n0, t0, bh);
        if (n0 + 64 < p.d.dv) tma_store_3d(map, stage + TILE, n0 + 64, t0, bh);
        tma_store_commit();
      }
    };
    bool ok = scale_chunk(0);
    for (int c = 0; c < NC; ++c) {
      const int g = c % GS, yb = c % NY, t0 = cg(c) * C;
      if (ok && c + 1 < NC) ok = scale_chunk(c + 1);
      ok = ok && mbar_wait_warp(&sm.yfull[yb], (c / NY) & 1, wc, W_O_Y);
      // the warps of emit() meet at barriers: all of them go on, or none does
      ok = !named_bar_or(2, 128, !ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = COL_D + 128 * yb;  // D^T (E^T)
      if (carry || (!BWD && !p.y)) {
        if (lane == 0) mbar_arrive(&sm.yfree[yb]);
      } else if constexpr (BWD) {
        emit(d, &tmY, sm.gates[g].be, t0, &sm.yfree[yb]);  // dV = beta E
      } else {
        emit(SPLIT ? COL_YS : d + 64, &tmY, nullptr, t0, &sm.yfree[yb]);
      }
      if (lane == 0) mbar_arrive(&sm.gempty[g]);
    }
    if (t == 0) tma_store_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

template <bool BWD, bool SPLIT>
static cudaError_t launch(const Args& a, bool sum, bool after, cudaStream_t st) {
  using L = Layout<BWD, SPLIT>;
  using gradlev::tc::make_map_bf16_3d;
  const Dims& d = a.d;
  const uint64_t N = chunks(d.T), kh = (uint64_t)d.B * d.Hk, bh = d.BH();
  const void* v = BWD ? a.dy : a.v;
  bf16* states = BWD ? a.dS : a.sv.S;
  const bf16* w = BWD ? a.sv.Wb : a.m.W;
  const bf16* t = BWD ? a.sv.PT : a.m.T0;
  bf16* dd = BWD ? a.E : a.sv.D;           // D or E
  void* yy = BWD ? a.dv_ : a.y;
  CUtensorMap mq, mk, mv, mw, mwl, mt, mtl, mp, ms, my, md;
  if (!make_map_bf16_3d(&mq, a.q, d.dk, d.T, kh, C) || !make_map_bf16_3d(&mk, a.k, d.dk, d.T, kh, C) ||
      !make_map_bf16_3d(&mv, v, d.dv, d.T, bh, C) || !make_map_bf16_3d(&mw, w, 128, N * C, bh, C) ||
      !make_map_bf16_3d(&mwl, SPLIT ? a.m.Wlo : w, 128, N * C, bh, C) ||
      !make_map_bf16_3d(&mt, t, C, N * C, bh, C) ||
      !make_map_bf16_3d(&mtl, SPLIT ? a.m.T0lo : t, C, N * C, bh, C) ||
      !make_map_bf16_3d(&mp, BWD ? t : a.m.Pb, C, N * C, bh, C) ||
      !make_map_bf16_3d(&ms, states ? (const void*)states : w, 128, states ? dvp(d) : N * C,
                        states ? bh * N : bh, 32) ||
      !make_map_bf16_3d(&my, yy ? yy : v, d.dv, d.T, bh, C) ||
      !gradlev::tc::make_map_bf16_3d_box(&md, dd ? (const void*)dd : w, dd ? C : 128,
                                         dd ? dvp(d) : N * C, dd ? bh * N : bh, 32, 32))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!bit || !(set.load() & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(
        walk_kernel<BWD, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::smem);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit);
  }
  const int ns = dvp(d) / 128, nseg = a.seg.nseg;
  WalkParams p{d, BWD ? a.sv.gates : a.m.gates, a.status, a.timeout_ns, a.S0, a.log_alpha,
               static_cast<const bf16*>(a.dST), a.ST, static_cast<bf16*>(a.dS0),
               static_cast<bf16*>(a.y), dd, states, nseg, a.seg.chunks, 0, nseg, ns, sum ? 0 : a.inject, sum,
               nseg > 1 ? a.init : nullptr, a.loc, a.M};
  unsigned grid = (unsigned)(bh * ns * nseg);
  if (sum) {  // forward: all segments but the last, with the identity; backward: all but the first
    p.seg0 = BWD ? 1 : 0;
    p.segs = nseg - 1;
    p.nsl = BWD ? ns : ns + 1;
    grid = (unsigned)(bh * p.nsl * p.segs);
  } else if (!BWD && nseg > 1 && a.sv.S) {
    grid += (unsigned)bh;  // the last segment's map, for the backward
  }
  if (after) {
    const cudaError_t e = launch_after(d, walk_kernel<BWD, SPLIT>, grid, kThreads, L::smem, st, mq, mk, mv,
                                       mw, mwl, mt, mtl, mp, ms, my, md, p);
    if (e != cudaSuccess) return e;
  } else {
    walk_kernel<BWD, SPLIT><<<grid, kThreads, L::smem, st>>>(mq, mk, mv, mw, mwl, mt, mtl, mp, ms, my,
                                                             md, p);
  }
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_walk(const Args& a, bool backward, bool split, bool sum, bool after,
                        cudaStream_t st) {
  if (backward) return launch<true, false>(a, sum, after, st);
  return split ? launch<false, true>(a, sum, after, st) : launch<false, false>(a, sum, after, st);
}

}  // namespace tc
}  // namespace delta
}  // namespace gradlev
