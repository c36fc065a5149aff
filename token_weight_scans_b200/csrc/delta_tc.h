// The gated delta rule on the tensor cores (tcgen05 / TMEM): bf16 I/O, d_k 24 to 128, d_v up
// to 256 (multiples of 8), chunks of 64 tokens. Formulas in delta.h.
//
// Three kernels:
//   prep  (delta_tc_prep.cu): per chunk, what does not depend on the state;
//   walk  (delta_tc_walk.cu): the state recurrence, forward or backward;
//   grad  (delta_tc_grad.cu): per chunk, the gradients of q, k and the gates.
// Few long scans are cut into segments that are walked at the same time (delta_tc_seg.cu).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"
#include "delta.h"

namespace gradlev {
namespace tc {
bool make_map_bf16_3d(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                      uint32_t box1);
bool make_map_bf16_3d_box(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                          uint32_t box0, uint32_t box1);
}

namespace delta {
namespace tc {

constexpr int C = 64;            // tokens per chunk
constexpr int TILE = C * 128;    // bytes of a [64 rows x 128 B] swizzled block
constexpr int BIG = 128 * 128;   // bytes of a [128 rows x 128 B] swizzled block
constexpr uint32_t LANE16 = 16u << 16;  // an M = 64 product in the upper 16 lanes of each 32

__host__ __device__ inline int chunks(int T) { return (T - 1) / C + 1; }

// d_k of 8 and 16: seven eighths of a tile's columns and more would be padding. They stay on the
// float32 kernels, which are the faster ones in small calls and in the forward (B8 H16 T4096 d_k 16
// d_v 64 575 against 600 us), though not with the gradients of large ones (2027 against 1014 us).
inline bool shape_ok(const Dims& d) { return d.bf16 && d.dk > 16 && d.dk <= 128 && d.dv <= 256; }

// The kernels work on 128 columns of d_k and whole slices of 128 rows of d_v. Narrower heads
// are padded with zeros by the TMA loads' bounds and cut off by those of the stores; only the
// buffers between the kernels hold the padded sizes.
__host__ __device__ inline int dvp(const Dims& d) { return d.dv <= 128 ? 128 : 256; }

using bf16 = __nv_bfloat16;

// Where keys are alike, the errors D of a chunk nearly cancel in P diag(beta) D and D^T K: each
// token takes back what the one before it wrote. A rounding of D, P, T0 or -T0 diag(G) K would be
// summed up over the chunk, unlike the values it sits on (y 1 to 5 %, dlog_alpha 20 % and more off
// where keys have a mean cosine of 0.9). So the triangular system is folded into the matrices that
// follow it, before anything is rounded. With R = V - diag(G) K S^T, the errors against the state
// at the chunk's start,
//   Kw = T0^T diag(beta w) K,   Pv = P diag(beta) T0,   Wq = scale diag(G) Q - Pv diag(G) K,
//   S <- G_C S + R^T Kw,        Y = Pv V + Wq S^T,      D = T0 R,
// and backwards
//   diag(beta) E = Pv^T dY + Kw dS^T,
//   dS <- G_C dS + dY^T Wq - (Kw dS^T)^T diag(G) K.
// A row of Kw, Pv or Wq is what is left of a token after all the ones that follow (precede) it, no
// longer than beta (scale) times a key, and its rounding counts like one of v itself: 2^-9 once.
// Only the gradients' per-token sums over a chunk (the grad kernel) need D and E apart, there as
// two bf16 each.
// beta is taken at least 2^-60 in size (bt): row j of Kw and column j of Pv carry it as a factor,
// and E_j is that of beta E divided by bt.
//
// Chunk-local matrices that the walks read, all bf16 with N*64 rows per (b, h):
//   Kw, Wq [64][128]; the remainders Kw2 for the forward, Wq2 for the backward; Kw3, what Kw2
//   leaves, for a forward whose last state is asked for;
//   Pv [64][64 | 64], its remainder behind it; T0 likewise, for the D that the backward needs.
struct Mats {
  bf16 *Kw = nullptr, *Kw2 = nullptr, *Kw3 = nullptr, *Wq = nullptr, *Wq2 = nullptr;
  bf16 *Pv = nullptr, *T0 = nullptr;
  float* gates = nullptr;   // [B*H][N] GateBlock
};

// The gates of a chunk as the kernels after prep read them (bulk copies of whole pieces: forward
// walk nG .. GC, gradients GC .. cb, backward walk GCb .. zb).
struct GateBlock {
  float nG[C];        // -G
  float z[C];         // beta / bt: 1, but 0 where beta = 0
  float GC, fac;      // fac != 0: M_ij = ra_i ca_j
  float pad[2];
  float bw[C];        // beta w
  float q[C];         // scale G
  float bG[C];        // -beta G
  float be[C];        // beta
  float ra[C], cb[C]; // cb = ca beta
  float GCb, padb[3];
  float zG[C];        // -G beta / bt
  float rb[C];        // 1 / bt
  float zb[C];        // beta / bt
};

// What the forward keeps for the backward: chunk-start states S [B*H][N][dvp][128], D^T
// [B*H][N][2][dvp][64] (bf16 and remainder, the tokens of a chunk contiguous, as the walk has
// them), Kw, Wq, Wq2, Pv and gates.
struct Saved {
  bf16 *S = nullptr, *D = nullptr, *Kw = nullptr, *Wq = nullptr, *Wq2 = nullptr, *Pv = nullptr;
  float *gates = nullptr, *M = nullptr;  // M: the segments' maps, with segments
};

// Segments of `chunks` chunks each (the last may be shorter).
struct SegPlan {
  int nseg, chunks;
};
SegPlan seg_plan(const Dims& d);
size_t saved_bytes(const Dims& d);
Saved saved_at(char* base, const Dims& d);
size_t fwd_scratch_bytes(const Dims& d);  // Mats
Mats mats_at(char* base, const Dims& d, bool saved);  // saved: what is not part of Saved
size_t bwd_scratch_bytes(const Dims& d);  // E and the chunk-end gradients of the state
size_t token_rows_bytes(const Dims& d);   // D^T or E^T, both parts

struct Args {
  Dims d;
  const void *q, *k, *v;
  const float *beta, *log_alpha;
  float scale;
  DeviceStatus* status;
  uint64_t timeout_ns;
  Mats m;
  Saved sv;                 // D, S null without checkpoints
  const float* S0 = nullptr;
  void* y = nullptr;
  float* ST = nullptr;
  const void* dy = nullptr;
  const void* dST = nullptr;
  bf16* E = nullptr;        // E^T, like D^T
  bf16* dS = nullptr;       // [B*H][N][dvp][128]: gradient of the chunk-end states
  void *dq = nullptr, *dk_ = nullptr, *dv_ = nullptr, *dbeta = nullptr, *dlog_alpha = nullptr;
  void* dS0 = nullptr;
  int inject = 0;           // test hook: the walk proper withholds one completion signal
  SegPlan seg{1, 1 << 30};
  float *loc = nullptr, *init = nullptr, *M = nullptr;  // with segments (WalkParams)
};

// Lays the segments' buffers out behind `at` (seg_bytes(d, own_M) bytes) and sets a.seg.
void set_segments(Args& a, char* at, float* M);
size_t seg_bytes(const Dims& d, bool own_M);

// A launch whose kernel waits by itself (grid_dep_wait, before it touches memory) for the one
// before it, so that its launch and setup overlap that one's end: 88.0 -> 82.9 us for training B2 H4
// T257. Calls of more than one wave of chunks launch in plain order: CTAs that move in early, one by
// one, cost them more than the gap between the kernels (B8 H16 T4096 1188 -> 1199 us).
// Nor do calls for the last state, whose kernels leave no room for the next one's CTAs beside them (T1000
// 80.7 -> 82.4 us).
inline bool launches_early(const Dims& d, bool last_state) {
  return !last_state && d.BH() * chunks(d.T) <= 3 * 148;
}
template <typename... P, typename... A>
cudaError_t launch_after(bool early, void (*kernel)(P...), unsigned grid, unsigned block, size_t smem,
                         cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}

// last_state: one that is asked for, with a bf16 more for its operands (delta_tc_walk.cu)
cudaError_t launch_prep(const Args& a, bool last_state, cudaStream_t st);
// after: a kernel of the same call is before it
cudaError_t launch_walk(const Args& a, bool backward, bool last_state, bool sum, bool after,
                        cudaStream_t st);
cudaError_t launch_combine(const Args& a, bool backward, cudaStream_t st);
cudaError_t launch_grad(const Args& a, cudaStream_t st);

cudaError_t run_fwd(const Args& a, cudaStream_t st);
cudaError_t run_bwd(const Args& a, cudaStream_t st);

// ---- gates of one chunk, one warp: lane l holds tokens l and l + 32.
struct GatePair {
  float be[2];        // beta
  float Lh[2], Ll[2]; // running sum of log alpha without the resets, high and low part
  int seg[2];         // resets up to and including the token
  float Lend, Lend_lo;
  int seg_end;
};

#ifdef __CUDACC__
struct RawGates { float la[2], be[2]; };
__device__ __forceinline__ RawGates load_gates(const float* beta, const float* log_alpha, size_t row,
                                               int t0, int T) {
  RawGates r;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int t = t0 + (threadIdx.x & 31) + 32 * k;
    r.la[k] = t < T ? log_alpha[row + t] : 0.f;
    r.be[k] = t < T ? beta[row + t] : 0.f;
  }
  return r;
}
__device__ __forceinline__ GatePair chunk_gates(const RawGates& raw) {
  const int lane = threadIdx.x & 31;
  GatePair g;
  // The running sum in 64-bit integers of 2^-40: exact, and no matter how strong the decays
  // are (a float32 sum would leave 1e-4 in the differences at L = -64 * 87). The two halves
  // of the chunk go side by side.
  long long L[2];
  unsigned m[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float la = raw.la[k];
    g.be[k] = raw.be[k];
    const bool reset = la < kResetLog;
    L[k] = reset ? 0 : __float2ll_rn(la * 0x1p40f);
    m[k] = __ballot_sync(0xffffffffu, reset);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u0 = __shfl_up_sync(0xffffffffu, L[0], o);
    const long long u1 = __shfl_up_sync(0xffffffffu, L[1], o);
    if (lane >= o) {
      L[0] += u0;
      L[1] += u1;
    }
  }
  L[1] += __shfl_sync(0xffffffffu, L[0], 31);
  const unsigned below = 0xffffffffu >> (31 - lane);
  g.seg[0] = __popc(m[0] & below);
  g.seg[1] = __popc(m[0]) + __popc(m[1] & below);
  g.seg_end = __popc(m[0]) + __popc(m[1]);
  const long long end = __shfl_sync(0xffffffffu, L[1], 31);
  auto split = [](long long v, float& hi, float& lo) {
    hi = __ll2float_rn(v);
    lo = __ll2float_rn(v - __float2ll_rn(hi)) * 0x1p-40f;
    hi *= 0x1p-40f;
  };
#pragma unroll
  for (int k = 0; k < 2; ++k) split(L[k], g.Lh[k], g.Ll[k]);
  split(end, g.Lend, g.Lend_lo);
  return g;
}
// G_i, w_i and G_C
__device__ __forceinline__ float gate_G(const GatePair& g, int k) {
  return g.seg[k] == 0 ? expf(g.Lh[k] + g.Ll[k]) : 0.f;
}
__device__ __forceinline__ float gate_w(const GatePair& g, int k) {
  return g.seg[k] == g.seg_end ? expf((g.Lend - g.Lh[k]) + (g.Lend_lo - g.Ll[k])) : 0.f;
}
__device__ __forceinline__ float gate_GC(const GatePair& g) {
  return g.seg_end == 0 ? expf(g.Lend + g.Lend_lo) : 0.f;
}
#endif

}  // namespace tc
}  // namespace delta
}  // namespace gradlev
