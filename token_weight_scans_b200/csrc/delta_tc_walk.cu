// Tensor-core gated delta rule: the state recurrence over the chunks of one scan, one CTA
// per (b, h, 128 rows of d_v). Matrices of struct Mats in delta_tc.h; everything on the
// state is transposed (rows of d_v in the 128 TMEM lanes, tokens or d_k in the columns),
// so that the two operands made from the previous product stay in tensor memory:
//
//   forward                                backward (chunks in reverse, S is dS)
//   R^T  = V^T - S (diag(G) K)^T           F^T  = S Kw^T
//   S    = G_C S + R^T Kw                  S    = G_C S + dY^T Wq - (beta / bt G F)^T K
//   Y^T  = V^T Pv^T + S Wq^T               bt E = F + Pv^T dY,  dV = beta E
//   D^T  = R^T T0^T (for the backward)
//
// The chain through a chunk is: S to bf16 (TMEM -> registers -> TMEM), the product with K (Kw),
// its result to bf16, the product with Kw (K). All else runs beside it: V^T of the next chunk
// (a product with the identity) and the outputs' products are issued into the gaps of the chain,
// and their results leave through an output warpgroup. One product of N = 128 takes S through K
// and Wq together; -G is applied to its result, so that K enters as it is.
//
// Every operand of the state that is not exact in bf16 comes as a sum of P bf16. Forward, P = 2:
// S, R and Kw (and Pv in Y, T0 in D). The gradients and y are then off by their own rounding and by
// that of what is multiplied once, Wq and the states that are kept: 1.7 to 2.4e-3, where one bf16
// each makes 2.4 to 3.3e-3. P = 3 where the last state is asked for: it is float32, and 16 bits
// would leave it 4e-6 off, not 8e-7. Backward, P = 2 for S, Wq and Pv; Kw and F are one.
//
// Warp roles (16): 0 and 3 TMA producers, 1 MMA issuer (owns TMEM), 2 copies the gates in,
// 4-11 two chain warpgroups (each half of the columns), which also leave S, D^T and E^T for
// the kernels after, 12-15 Y (dV): 16-lane TMEM loads in the layout of 8 x 8 fragments, transposed on
// the way to shared memory (stmatrix) so that tokens become rows, and TMA stores. D^T and E^T stay as
// they are, a chunk's tokens contiguous, in two bf16 each.
//
// Measured (B8 H16 T4096 d 128, 128 CTAs of 64 chunks): forward 270 us, backward 226 us, of
// 3080 and 2830 bytes per token: 6.0 and 6.5 TB/s, near the measured copy bandwidth (6.47). Where HBM
// does not bound it, a chunk takes 2.5 us (forward without outputs), 3.6 us with P = 3: the chain, two
// products of P or P (P + 1) / 2 parts each and two passes of the state or R through registers. S, D
// and E go through shared memory: stored from registers, 16 bytes per row and instruction, the walks
// of d_v 256 took a third longer.
//
// Each chunk's tiles come in groups that are done with at different times: V (dY); K (Kw) with Wq;
// Kw (K); Pv; T0. The first two have two places each; the others, for which a chunk's time is enough
// to come, have one.
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
constexpr uint32_t COL_SH = 128;   // bf16 state, 64 for each part
// Over it, once the products with K have read it: the bf16 operand of the update, 32 for each part
// (R with 0 where beta = 0, backward -G F), and behind it R in two parts, for D
constexpr uint32_t COL_U = 128;
// Accumulators. Forward: V^T, then D^T in its place (P = 2: two such), S K^T and Y^T. Backward: two
// pairs of Pv^T dY and F.
constexpr uint32_t COL_SK = 384, COL_Y = 448;
constexpr uint32_t COL_P = 256;
template <int P> constexpr uint32_t COL_DB = COL_U + 32 * P;
template <int P> constexpr uint32_t COL_V = P == 2 ? 256 : 320;

// A chunk's gates: the piece of GateBlock that the direction needs, as it lies there.
template <bool BWD> struct GateSlot;
template <> struct GateSlot<false> {
  float nG[C], u[C], GC, pad[3];        // nG .. GC
  static constexpr size_t offset = offsetof(GateBlock, nG);
};
template <> struct GateSlot<true> {
  float GC, pad[3], u[C], rb[C], z[C];  // GCb .. zb
  static constexpr size_t offset = offsetof(GateBlock, GCb);
};
static_assert(sizeof(GateSlot<false>) % 16 == 0 && sizeof(GateSlot<true>) % 16 == 0 &&
              offsetof(GateBlock, GCb) % 16 == 0 && sizeof(GateBlock) % 16 == 0, "bulk copies");

template <bool BWD>
struct Bars {
  GateSlot<BWD> gates[GS];
  uint64_t full[3][NS], empty[3][NS];   // per group of tiles
  uint64_t gfull[GS], gempty[GS];
  uint64_t sready[2];                   // in two halves of each warp's columns
  uint64_t sscaled, dfull, uready, sfull, done;
  uint64_t pfull, pempty, tfull, tempty;  // Pv; T0
  uint64_t ddone, dfree[2];             // D^T
  uint64_t yfull[2], yfree[2];          // per accumulator (pair)
  uint32_t tmem_base;
  int abort;
};
enum { VD = 0, KQ = 1, UP = 2 };

// VD: V (dY). KQ: per 64 columns of d_k the K (Kw) tile and the Wq tile next to each other (128 rows
// of one operand), backward also the remainder of Wq. UP: Kw in its parts (K).
template <bool BWD, int P>
struct Layout {
  static constexpr int w = 0, q = TILE;
  static constexpr int wq = BWD ? 3 * TILE : 2 * TILE;  // from one k-block to the next
  static constexpr int vd_bytes = 2 * TILE, kq_bytes = 2 * wq;
  static constexpr int up_bytes = BWD ? 2 * TILE : 2 * P * TILE;
  static constexpr int kq0 = NS * vd_bytes, up = kq0 + NS * kq_bytes;
  // Pv, forward T0, with their remainders; forward the identity
  static constexpr int pv = up + up_bytes, t0 = pv + 2 * TILE;
  static constexpr int id = t0 + (BWD ? 0 : 2 * TILE);
  // S, and after it D^T (E^T), through shared memory and TMA: 4 KB for each warp of the chain
  static constexpr bool staged = P == 2;
  static constexpr int stage_s = id + (BWD ? 0 : TILE), stage_o = stage_s + (staged ? 2 * BIG : 0);
  static constexpr int bars = stage_o + 2 * TILE;
  static constexpr size_t smem = bars + sizeof(Bars<BWD>) + 1024;
  static_assert(smem <= 227 * 1024, "over the shared memory of a CTA");
  static constexpr int vd(int s) { return s * vd_bytes; }
  static constexpr int kq(int s) { return kq0 + s * kq_bytes; }
};

enum : uint32_t {
  W_TMA = 0x901, W_TMA_DRAIN, W_FULL = 0x911, W_SREADY, W_UREADY, W_YFREE, W_DFREE, W_DONE,
  W_GATE = 0x921, W_PV, W_T0, W_C_SFULL = 0x931, W_C_DFULL, W_C_DDONE, W_C_GATE, W_O_GATE = 0x941, W_O_Y,
  W_O_DDONE,
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
  bf16* D;               // forward: D^T, backward: E^T, two parts (null: not kept)
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

__device__ __forceinline__ void st_tmem16(uint32_t col, const uint32_t (&r)[16]) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
  tmem_st16(col, v);
}
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t hi) {
  return pack_bf16(a - bf16_lo(hi), b - bf16_hi(hi));
}

// The gates that only one direction has.
__device__ __forceinline__ const float* gate_nG(const GateSlot<false>& g) { return g.nG; }
__device__ __forceinline__ const float* gate_nG(const GateSlot<true>&) { return nullptr; }
__device__ __forceinline__ const float* gate_rb(const GateSlot<true>& g) { return g.rb; }
__device__ __forceinline__ const float* gate_rb(const GateSlot<false>&) { return nullptr; }
__device__ __forceinline__ const float* gate_z(const GateSlot<true>& g) { return g.z; }

// N values as two bf16, the remainders `apart` elements behind.
template <int N>
__device__ __forceinline__ void store_split(bf16* out, size_t apart, const float (&v)[N]) {
#pragma unroll
  for (int cc = 0; cc < N / 8; ++cc) {
    uint32_t hi[4], rest[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      hi[e] = pack_bf16(v[8 * cc + 2 * e], v[8 * cc + 2 * e + 1]);
      rest[e] = pack_rest(v[8 * cc + 2 * e], v[8 * cc + 2 * e + 1], hi[e]);
    }
    *reinterpret_cast<uint4*>(out + 8 * cc) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(out + apart + 8 * cc) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
  }
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

template <bool BWD, int P>
__global__ void __launch_bounds__(kThreads, 1)
    walk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ CUtensorMap tmKw, const __grid_constant__ CUtensorMap tmKw2,
                const __grid_constant__ CUtensorMap tmKw3, const __grid_constant__ CUtensorMap tmWq,
                const __grid_constant__ CUtensorMap tmWq2,
                const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmT,
                const __grid_constant__ CUtensorMap tmS, const __grid_constant__ CUtensorMap tmY,
                const __grid_constant__ CUtensorMap tmD, WalkParams p) {
  using L = Layout<BWD, P>;
  constexpr int NY = BWD ? 2 : 1, NV = P == 2 ? 2 : 1;  // places of Y (pairs); of V and D
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
  const bool outputs = !BWD && !carry && p.y;        // the forward's products for Y
  const bool errors = !BWD && !carry && p.D;         // and those for D
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
    }
    for (int g = 0; g < GS; ++g) {
      mbar_init(&sm.gfull[g], 1);
      mbar_init(&sm.gempty[g], BWD ? 12 : 8);  // the chain's 8 warps, backward the 4 of dV
    }
    mbar_init(&sm.sready[0], 8);
    mbar_init(&sm.sready[1], 8);
    mbar_init(&sm.sscaled, 8);
    mbar_init(&sm.dfull, 1);
    mbar_init(&sm.uready, 8);
    mbar_init(&sm.sfull, 1);
    mbar_init(&sm.done, 1);
    mbar_init(&sm.pfull, 1);
    mbar_init(&sm.pempty, 1);
    mbar_init(&sm.tfull, 1);
    mbar_init(&sm.tempty, 1);
    mbar_init(&sm.ddone, 1);
    for (int y = 0; y < 2; ++y) {
      mbar_init(&sm.yfull[y], 1);
      mbar_init(&sm.yfree[y], 4);
      mbar_init(&sm.dfree[y], 8);
    }
    fence_mbar_init();
  }
  if (!BWD) {  // the identity, 16 bytes per thread
    const int r = threadIdx.x >> 3, c = threadIdx.x & 7, e = r & 7;
    const uint32_t one = (r >> 3) == c ? 0x3F80u << (16 * (e & 1)) : 0u;  // bf16
    st_shared_v4(smem_u32(base + L::id) + sw128_off(r, c), e >> 1 == 0 ? one : 0u, e >> 1 == 1 ? one : 0u,
                 e >> 1 == 2 ? one : 0u, e >> 1 == 3 ? one : 0u);
    fence_proxy_async_smem();
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
    // warp 0: V (dY, with Pv), and Kw (K); warp 3: K (Kw) with Wq
    if (lane == 0) {
      int issued[3] = {0, 0, 0};
      auto places = [](int r) { return r == UP ? 1 : NS; };
      auto open = [&](int r, int c, int bytes) -> bool {
        const int n = places(r);
        if (!mbar_wait(&sm.empty[r][c % n], ((c / n) & 1) ^ 1, wc, W_TMA)) return false;
        mbar_arrive_expect_tx(&sm.full[r][c % n], bytes);
        issued[r] = c + 1;
        return true;
      };
      const bool wq = BWD || outputs;
      for (int c = 0; c < NC; ++c) {
        const int s = c % NS, t0 = cg(c) * C;
        if (warp == 0) {
          uint8_t* a = base + L::vd(s);
          uint64_t* f = &sm.full[VD][s];
          if (!open(VD, c, L::vd_bytes)) break;
          const int tv = ident ? N * C : t0;  // past the last token: zeros
          tma_load_3d(a, &tmV, f, n0, tv, bh);
          tma_load_3d(a + TILE, &tmV, f, n0 + 64, tv, bh);
          a = base + L::up;
          f = &sm.full[UP][0];
          if (!open(UP, c, L::up_bytes)) break;
          for (int kb = 0; kb < 2; ++kb) {
            tma_load_3d(a + kb * TILE, BWD ? &tmK : &tmKw, f, 64 * kb, t0, BWD ? kh : bh);
            if (!BWD) tma_load_3d(a + (2 + kb) * TILE, &tmKw2, f, 64 * kb, t0, bh);
            if (!BWD && P > 2) tma_load_3d(a + (4 + kb) * TILE, &tmKw3, f, 64 * kb, t0, bh);
          }
        } else {
          uint8_t* a = base + L::kq(s);
          uint64_t* f = &sm.full[KQ][s];
          if (!open(KQ, c, wq ? L::kq_bytes : 2 * TILE)) break;
          for (int kb = 0; kb < 2; ++kb, a += L::wq) {
            tma_load_3d(a + L::w, BWD ? &tmKw : &tmK, f, 64 * kb, t0, BWD ? bh : kh);
            if (wq) tma_load_3d(a + L::q, &tmWq, f, 64 * kb, t0, bh);
            if (BWD) tma_load_3d(a + L::q + TILE, &tmWq2, f, 64 * kb, t0, bh);
          }
        }
      }
      // teardown: every load issued has landed
      for (int r = 0; r < 3; ++r)
        for (int n = places(r), c = issued[r] > n ? issued[r] - n : 0; c < issued[r]; ++c)
          mbar_drain(&sm.full[r][c % n], (c / n) & 1, wc, W_TMA_DRAIN);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t id_v = idesc_bf16(128, 64, true, BWD);       // V^T I, V^T Pv^T, dY^T Pv
      const uint32_t id_w = idesc_bf16(128, 64, false, false);    // S K^T, S Kw^T, R^T T0^T
      const uint32_t id_wq = idesc_bf16(128, 128, false, false);  // S [K; Wq]^T
      const uint32_t id_u = idesc_bf16(128, 128, false, true);    // R^T Kw, F^T K
      const uint32_t id_o = idesc_bf16(128, 128, true, true);     // dY^T Wq
      // d (+)= (V or dY)^T b, b [64 x 64] at shared address b
      auto from_v = [&](uint32_t d, int c, uint32_t b, bool on) {
        const uint32_t sv = smem_u32(base + L::vd(c % NS));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16(d, desc_at(sw128_desc(sv, TILE, 1024), kk * 2048),
                    desc_at(sw128_desc(b, BWD ? TILE : 16, 1024), BWD ? kk * 2048 : kk * 32), id_v,
                    on || kk > 0);
      };
      const uint32_t s_id = smem_u32(base + L::id), s_pv = smem_u32(base + L::pv);
      const uint32_t s_t0 = smem_u32(base + L::t0);
      // What of chunk c needs no state. Its accumulators are free once the chain has read R
      // (uready, waited by then) and D, and the outputs have been taken.
      auto first = [&](int c) -> bool {
        if (!mbar_wait(&sm.full[VD][c % NS], (c / NS) & 1, wc, W_FULL)) return false;
        if (BWD) {
          if (!mbar_wait(&sm.yfree[c & 1], ((c >> 1) & 1) ^ 1, wc, W_YFREE)) return false;
          if (!carry) {
            if (!mbar_wait(&sm.pfull, c & 1, wc, W_FULL)) return false;
            tc_fence_after();
            const uint32_t d = tb + COL_P + 128 * (c & 1);
            from_v(d, c, s_pv, false);
            from_v(d, c, s_pv + TILE, true);
            umma_commit(&sm.pempty);
          }
          return true;
        }
        if (errors) {
          if (P == 2 ? !mbar_wait(&sm.dfree[c % NV], ((c / NV) & 1) ^ 1, wc, W_DFREE)
                     : !mbar_wait(&sm.yfree[0], (c & 1) ^ 1, wc, W_YFREE))
            return false;
        }
        tc_fence_after();
        from_v(tb + COL_V<P> + 64 * (c % NV), c, s_id, false);
        return true;
      };
      bool ok = first(0);
      for (int c = 0; c < NC && ok; ++c) {
        const int s = c % NS;
        const uint32_t st = smem_u32(base + L::kq(s)), sk = smem_u32(base + L::up);
        // S K^T and Y^T behind it; F^T
        const uint32_t d = BWD ? tb + COL_P + 128 * (c & 1) + 64 : tb + COL_SK;
        if (!mbar_wait(&sm.full[KQ][s], (c / NS) & 1, wc, W_FULL)) break;
        bool got = !outputs || mbar_wait(&sm.yfree[0], (c & 1) ^ 1, wc, W_YFREE);
        // the K steps in the order in which the two warpgroups convert S, so that the products
        // of the first half run while the second is converted
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          got = got && mbar_wait(&sm.sready[half], c & 1, wc, W_SREADY);
          if (!got) break;
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int kk = 4 * (j >> 1) + 2 * half + (j & 1);
            const uint64_t kq = desc_at(sw128_desc(st + L::w, 16, 1024), (kk >> 2) * L::wq + (kk & 3) * 32);
#pragma unroll
            for (int i = 0; i < P; ++i)
              umma_bf16_tmem_a(d, tb + COL_SH + 64 * i + 8 * kk, kq, outputs && i < 2 ? id_wq : id_w,
                               half + j + i > 0);
          }
        }
        if (!got) break;
        if (!(p.inject && c == 1)) umma_commit(&sm.dfull);
        if (BWD) {
          umma_commit(&sm.yfull[c & 1]);
          if (!mbar_wait(&sm.sscaled, c & 1, wc, W_SREADY)) break;
          tc_fence_after();
          const uint32_t sv = smem_u32(base + L::vd(s));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {  // S += dY^T Wq
            const uint64_t av = desc_at(sw128_desc(sv, TILE, 1024), kk * 2048);
            const uint64_t bq = desc_at(sw128_desc(st + L::q, L::wq, 1024), kk * 2048);
            umma_bf16(tb + COL_S, av, bq, id_o, 1);
            umma_bf16(tb + COL_S, av, desc_at(bq, TILE), id_o, 1);
          }
        } else if (outputs) {  // Y^T += V^T Pv^T
          if (!mbar_wait(&sm.pfull, c & 1, wc, W_FULL)) break;
          tc_fence_after();
          from_v(tb + COL_Y, c, s_pv, true);
          from_v(tb + COL_Y, c, s_pv + TILE, true);
          umma_commit(&sm.pempty);
          umma_commit(&sm.yfull[0]);
        }
        umma_commit(&sm.empty[VD][s]);
        umma_commit(&sm.empty[KQ][s]);
        if (!mbar_wait(&sm.full[UP][0], c & 1, wc, W_FULL)) break;
        if (!mbar_wait(&sm.uready, c & 1, wc, W_UREADY)) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {  // S += U^T Kw, parts i and j down to 2^-8 of the last
#pragma unroll
          for (int i = 0; i < (BWD ? 1 : P); ++i)
#pragma unroll
            for (int j = 0; j < (BWD ? 1 : P); ++j)
              if (i + j < P)
                umma_bf16_tmem_a(tb + COL_S, tb + COL_U + 32 * i + 8 * kk,
                                 desc_at(sw128_desc(sk + 2 * j * TILE, TILE, 1024), kk * 2048), id_u, 1);
        }
        umma_commit(&sm.sfull);
        umma_commit(&sm.empty[UP][0]);
        if (!BWD && errors) {  // D^T = R^T T0^T
          if (!mbar_wait(&sm.tfull, c & 1, wc, W_FULL)) break;
          tc_fence_after();
          const uint32_t e = tb + COL_V<P> + 64 * (c % NV);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t hi = desc_at(sw128_desc(s_t0, 16, 1024), kk * 32);
            umma_bf16_tmem_a(e, tb + COL_DB<P> + 8 * kk, hi, id_w, kk > 0);
            umma_bf16_tmem_a(e, tb + COL_DB<P> + 8 * kk, desc_at(hi, TILE), id_w, 1);
            umma_bf16_tmem_a(e, tb + COL_DB<P> + 32 + 8 * kk, hi, id_w, 1);
          }
          umma_commit(&sm.ddone);
          umma_commit(&sm.tempty);
        }
        if (c + 1 < NC) ok = first(c + 1);
      }
      umma_commit(&sm.done);
      mbar_drain(&sm.done, 0, wc, W_DONE);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ gates
    if (lane == 0) {
      const char* src = reinterpret_cast<const char*>(p.gates) + GateSlot<BWD>::offset;
      int issued = 0, loaded = 0;
      auto gates = [&](int c) -> bool {
        const int g = c % GS;
        if (!mbar_wait(&sm.gempty[g], ((c / GS) & 1) ^ 1, wc, W_GATE)) return false;
        mbar_arrive_expect_tx(&sm.gfull[g], sizeof(GateSlot<BWD>));
        bulk_load(&sm.gates[g], src + ((size_t)bh * N + cg(c)) * sizeof(GateBlock),
                  sizeof(GateSlot<BWD>), &sm.gfull[g]);
        issued = c + 1;
        return true;
      };
      // Pv and T0 wait for the chunk before, so the gates go two chunks ahead of them
      auto pair = [&](int at, const CUtensorMap* map, uint64_t* full, uint64_t* empty, int c, uint32_t where) {
        if (!mbar_wait(empty, (c & 1) ^ 1, wc, where)) return false;
        mbar_arrive_expect_tx(full, 2 * TILE);
        tma_load_3d(base + at, map, full, 0, cg(c) * C, bh);
        tma_load_3d(base + at + TILE, map, full, 64, cg(c) * C, bh);
        return true;
      };
      int pvs = 0;
      bool ok = gates(0) && (NC < 2 || gates(1));
      for (int c = 0; c < NC && ok; ++c) {
        if (BWD ? !carry : outputs) {
          if (!pair(L::pv, &tmP, &sm.pfull, &sm.pempty, c, W_PV)) break;
          pvs = c + 1;
        }
        if (!BWD && errors) {
          if (!pair(L::t0, &tmT, &sm.tfull, &sm.tempty, c, W_T0)) break;
          loaded = c + 1;
        }
        if (c + 2 < NC) ok = gates(c + 2);
      }
      for (int c = issued > GS ? issued - GS : 0; c < issued; ++c)
        mbar_drain(&sm.gfull[c % GS], (c / GS) & 1, wc, W_TMA_DRAIN);
      if (pvs) mbar_drain(&sm.pfull, (pvs - 1) & 1, wc, W_TMA_DRAIN);
      if (loaded) mbar_drain(&sm.tfull, (loaded - 1) & 1, wc, W_TMA_DRAIN);
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
    // 32 tokens of this row of D (E) as two bf16, the whole warp: through the warp's part of the
    // buffer that S went through, 64-byte rows and swizzle
    auto leave = [&](const float (&x)[32], int n) {
      if (lane == 0) tma_store_wait_read_n<0>();
      __syncwarp();
      uint8_t* const part = base + L::stage_s + (warp - 4) * 4096;
      const uint32_t at = smem_u32(part) + lane * 64;
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        uint32_t hi[4], rest[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          hi[e] = pack_bf16(x[8 * cc + 2 * e], x[8 * cc + 2 * e + 1]);
          rest[e] = pack_rest(x[8 * cc + 2 * e], x[8 * cc + 2 * e + 1], hi[e]);
        }
        const uint32_t off = (cc ^ ((lane >> 1) & 3)) << 4;
        st_shared_v4(at + off, hi[0], hi[1], hi[2], hi[3]);
        st_shared_v4(at + 2048 + off, rest[0], rest[1], rest[2], rest[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(&tmD, part, 32 * hh, n0 + 32 * q, bh * N + n);
        tma_store_3d(&tmD, part + 2048, 32 * hh, rows + n0 + 32 * q, bh * N + n);
        tma_store_commit();
      }
    };
    // D of chunk c, once its product is done, and its place for the chunk after the next
    auto leave_D = [&](int c) {
      float x[32];
      tmem_ld32(tb + COL_V<P> + 64 * (c % NV) + lo + 32 * hh, x);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.dfree[c % NV]);
      leave(x, cg(c));
    };
    constexpr bool chain_D = !BWD && P == 2;
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
      // 32 columns at a time (registers), each half as it is ready
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float v[32];
        tmem_ld32(at + 32 * hf, v);
        tmem_ld_wait();
        if (!BWD && errors && hf == 0 && c > 0)  // D's product has read what the parts go over
          ok = mbar_wait_warp(&sm.ddone, (c - 1) & 1, wc, W_C_DDONE);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < P; ++i) {
          uint32_t part[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            part[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
            if (i == 0) pk[16 * hf + e] = part[e];
            v[2 * e] -= bf16_lo(part[e]);
            v[2 * e + 1] -= bf16_hi(part[e]);
          }
          st_tmem16(tb + COL_SH + 64 * i + lo + 32 * hh + 16 * hf, part);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.sready[hf]);
      }
      if (!ok) break;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {  // the decay, read again: not before the update (dY^T Wq)
        float v[32];
        tmem_ld32(at + 32 * hf, v);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] *= GC;
        tmem_st32(at + 32 * hf, v);
      }
      if (BWD) {
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.sscaled);
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
      auto factors = [&](const float* f) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 x = *reinterpret_cast<const float4*>(f + 32 * hh + e);
          uf[e] = x.x;
          uf[e + 1] = x.y;
          uf[e + 2] = x.z;
          uf[e + 3] = x.w;
        }
      };
      factors(BWD ? gs.u : gate_nG(gs));
      ok = mbar_wait_warp(&sm.dfull, c & 1, wc, W_C_DFULL);
      if (!ok) break;
      tc_fence_after();
      float v[32];  // R, or F
      // backward: Pv^T dY, and F behind it
      const uint32_t acc = tb + (BWD ? COL_P + 128 * (c & 1) : COL_SK) + lo + 32 * hh;
      tmem_ld32(BWD ? acc + 64 : tb + COL_V<P> + 64 * (c % NV) + lo + 32 * hh, v);
      if constexpr (!BWD) {
        float w[32];
        tmem_ld32(acc, w);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = fmaf(uf[e], w[e], v[e]);
        factors(gs.u);
      } else {
        tmem_ld_wait();
      }
      // v times the factors if given, in `parts` bf16 from column `col` on
      auto put_parts = [&](uint32_t col, int parts, bool times) {
        float x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = times ? v[e] * uf[e] : v[e];
#pragma unroll
        for (int i = 0; i < parts; ++i) {
          uint32_t part[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            part[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
            x[2 * e] -= bf16_lo(part[e]);
            x[2 * e + 1] -= bf16_hi(part[e]);
          }
          st_tmem16(tb + col + 32 * i + lo + 16 * hh, part);
        }
      };
      put_parts(COL_U, BWD ? 1 : P, true);
      if (!BWD && errors) put_parts(COL_DB<P>, 2, false);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.uready);
      if (BWD && !carry) {  // E = (F + Pv^T dY) / bt
        float w[32];
        factors(gate_rb(gs));
        tmem_ld32(acc, w);
        tmem_ld_wait();
        tc_fence_before();
#pragma unroll
        for (int e = 0; e < 32; ++e) w[e] = (w[e] + v[e]) * uf[e];
        leave(w, n);
      }
      // D of the chunk before: its product was issued before the one that dfull stands for
      if (chain_D && errors && c > 0) leave_D(c - 1);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.gempty[g]);
    }
    if (chain_D && errors && ok && mbar_wait_warp(&sm.ddone, (NC - 1) & 1, wc, W_C_DDONE)) {
      tc_fence_after();
      leave_D(NC - 1);
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
    // ------------------------------------------------------------ outputs
    const int q = warp & 3, t = threadIdx.x & 127;
    const uint32_t lo = (uint32_t)(32 * q) << 16;
    // 128 rows x 64 tokens at TMEM column `col` (backward: the sum of those and the 64 behind them) to
    // a [64 tokens x 128] tile of `map`, times factor[token] if given
    uint8_t* const stage = base + L::stage_o;
    const uint32_t tile = smem_u32(stage);
    auto emit = [&](uint32_t col, const CUtensorMap* map, const float* factor, int t0, uint64_t* after) {
      if (t == 0) tma_store_wait_read_n<0>();  // the tile's last store
      named_bar_sync(1, 128);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float v[32];
        tmem_ld_frag64(tb + col + lo + hf * LANE16, v);
        if constexpr (BWD) {
          float w[32];
          tmem_ld_frag64(tb + col + 64 + lo + hf * LANE16, w);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] += w[e];
        } else {
          tmem_ld_wait();
        }
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
    const bool own_D = !BWD && P == 3 && errors;  // (P = 2: the chain)
    bool ok = true;
    for (int c = 0; c < NC && (BWD || outputs || own_D); ++c) {
      const int g = c % GS, yb = c % NY, t0 = cg(c) * C;
      if (BWD) ok = ok && mbar_wait_warp(&sm.gfull[g], (c / GS) & 1, wc, W_O_GATE);
      if (BWD || outputs) ok = ok && mbar_wait_warp(&sm.yfull[yb], (c / NY) & 1, wc, W_O_Y);
      if (own_D) ok = ok && mbar_wait_warp(&sm.ddone, c & 1, wc, W_O_DDONE);
      // the warps of emit() meet at barriers: all of them go on, or none does
      ok = !named_bar_or(2, 128, !ok);
      if (!ok) break;
      tc_fence_after();
      if (own_D) {  // two bf16: a row of 64 tokens per thread
        bf16* const out = p.D + (((size_t)bh * N + cg(c)) * 2 * dvp(p.d) + n0 + 32 * q + lane) * C;
#pragma unroll
        for (int hf = 0; hf < 4; ++hf) {
          float v[16];
          tmem_ld16(tb + COL_V<P> + lo + 16 * hf, v);
          tmem_ld_wait();
          store_split<16>(out + 16 * hf, (size_t)dvp(p.d) * C, v);
        }
      }
      if (carry || (!BWD && !outputs)) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.yfree[yb]);
      } else if constexpr (BWD) {
        emit(COL_P + 128 * yb, &tmY, gate_z(sm.gates[g]), t0, &sm.yfree[yb]);  // dV = beta E
      } else {
        emit(COL_Y, &tmY, nullptr, t0, &sm.yfree[yb]);
      }
      __syncwarp();
      if (BWD && lane == 0) mbar_arrive(&sm.gempty[g]);
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

template <bool BWD, int P>
static cudaError_t launch(const Args& a, bool sum, bool after, cudaStream_t st) {
  using L = Layout<BWD, P>;
  using gradlev::tc::make_map_bf16_3d;
  const Dims& d = a.d;
  const uint64_t N = chunks(d.T), kh = (uint64_t)d.B * d.Hk, bh = d.BH();
  const void* v = BWD ? a.dy : a.v;
  bf16* states = BWD ? a.dS : a.sv.S;
  const Mats& m = a.m;
  bf16* dd = BWD ? a.E : a.sv.D;           // D or E
  void* yy = BWD ? a.dv_ : a.y;
  CUtensorMap mk, mv, mw, mw2, mw3, mq, mq2, mp, mt, ms, my, md;
  auto mat = [&](CUtensorMap* t, const bf16* x) { return make_map_bf16_3d(t, x, 128, N * C, bh, C); };
  if (!make_map_bf16_3d(&mk, a.k, d.dk, d.T, kh, C) || !make_map_bf16_3d(&mv, v, d.dv, d.T, bh, C) ||
      !mat(&mw, m.Kw) || !mat(&mw2, BWD ? m.Kw : m.Kw2) || !mat(&mw3, P == 3 ? m.Kw3 : m.Kw) ||
      !mat(&mq, m.Wq) || !mat(&mq2, BWD ? m.Wq2 : m.Wq) || !mat(&mp, m.Pv) ||
      !mat(&mt, !BWD && dd ? m.T0 : m.Pv) ||
      !make_map_bf16_3d(&ms, states ? states : m.Kw, 128, states ? dvp(d) : N * C,
                        states ? bh * N : bh, 32) ||
      !make_map_bf16_3d(&my, yy ? yy : v, d.dv, d.T, bh, C) ||
      !gradlev::tc::make_map_bf16_3d_box(&md, dd ? dd : m.Kw, dd ? C : 128, dd ? 2 * dvp(d) : N * C,
                                         dd ? bh * N : bh, 32, 32))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!bit || !(set.load() & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(
        walk_kernel<BWD, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::smem);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit);
  }
  const int ns = dvp(d) / 128, nseg = a.seg.nseg;
  WalkParams p{d, m.gates, a.status, a.timeout_ns, a.S0, a.log_alpha,
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
    const cudaError_t e = launch_after(launches_early(d, a.ST != nullptr), walk_kernel<BWD, P>, grid, kThreads, L::smem, st, mk, mv, mw, mw2,
                                       mw3, mq, mq2, mp, mt, ms, my, md, p);
    if (e != cudaSuccess) return e;
  } else {
    walk_kernel<BWD, P><<<grid, kThreads, L::smem, st>>>(mk, mv, mw, mw2, mw3, mq, mq2, mp, mt, ms, my, md, p);
  }
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_walk(const Args& a, bool backward, bool last_state, bool sum, bool after,
                        cudaStream_t st) {
  if (backward) return launch<true, 2>(a, sum, after, st);
  return last_state ? launch<false, 3>(a, sum, after, st) : launch<false, 2>(a, sum, after, st);
}

}  // namespace tc
}  // namespace delta
}  // namespace gradlev
