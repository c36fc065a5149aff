// Internal interface of the gated delta rule (gradlev_delta_*): the argument blocks
// of its kernel families and the layout of what they keep between passes.
//
// Per (b, value head h), with the key head h / (H / Hk) and S [d_v, d_k]:
//   S' = a_t S_{t-1},  e_t = v_t - S' k_t,  S_t = S' + beta_t e_t k_t^T,
//   y_t = scale S_t q_t,                    a_t = exp(log_alpha_t).
//
// Within a chunk of C tokens, with L the running sum of log_alpha, G_i = exp(L_i),
// M_ij = exp(L_i - L_j) (j <= i), S the state before the chunk, and the rows of K, Q,
// V the tokens':
//   A_ij = M_ij k_i.k_j (j < i),   Z = (I + A diag(beta))^-1 A   (strictly lower)
//   R = V - diag(G) K S^T,         D = R - Z diag(beta) R        (row t is e_t)
//   P_ij = scale M_ij q_i.k_j (j <= i)
//   Y = scale diag(G) Q S^T + P diag(beta) D
//   S <- G_C S + D^T diag(beta w) K,   w_j = exp(L_{C-1} - L_j)
// and backwards, with dS the gradient of the state after the chunk:
//   F = P^T dY + diag(w) K dS^T,   E = F - Z^T diag(beta) F,     dV = diag(beta) E
//   dS <- G_C dS + dY^T diag(scale G) Q - E^T diag(beta G) K
//   X_ij = scale M_ij beta_j dy_i.D_j (j <= i),  Y_ij = M_ij beta_i beta_j E_i.D_j (j < i)
//   dQ = scale diag(G) dY S + X K
//   dK = -diag(beta G) E S + X^T Q + diag(beta w) D dS - (Y + Y^T) K
//   dbeta_i = E_i.D_i
//   dlog_alpha_t = sum_{i>=t} (x_i - y_i) + sum_{j<t} z_j + G_C <dS, S>
//                  + sum_{i>=t>j} (X_ij q_i.k_j - Y_ij k_i.k_j),
//     x_i = scale G_i q_i.(S^T dy_i), y_i = beta_i G_i k_i.(S^T E_i),
//     z_j = beta_j w_j k_j.(dS^T D_j).
// Z rather than an inverse is kept: both inverses the two directions need,
// (I + A diag(beta))^-1 = I - Z diag(beta) and (I + diag(beta) A)^-1 = I - diag(beta) Z,
// follow from it also where beta = 0.
//
// log_alpha = -inf (a_t = 0) starts a new sequence. exp of a difference of infinities
// has no value, so resets stay out of L and are counted instead: M_ij, G_i and w_j are
// zero across a reset. A log_alpha below kResetLog underflows float32 and counts as one.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"

namespace gradlev {
namespace delta {

constexpr float kResetLog = -87.f;

struct Dims {
  int B, H, Hk, T, dk, dv;
  bool bf16;
  size_t BH() const { return (size_t)B * H; }
};

// ---- float32 kernels (products of split tf32 operands), chunks of 32 tokens
namespace ffma {

constexpr int C = 32;

// What the forward leaves for the backward, all float32:
//   S [B*H][N][dv][dk] chunk-start states, D [B*H][T][dv], Z and P [B*H][N][C][C], gates
//   [B*H][N] WalkGates.
struct Saved {
  float *S, *D, *Z, *P, *gates;
};
// A chunk's gates as the walks copy them in.
struct WalkGates {
  float beta[C], G[C], w[C];
  float GC, pad[3];
};
__host__ __device__ inline int chunks(int T) { return (T - 1) / C + 1; }
size_t saved_bytes(const Dims& d, bool states);  // states = false: Z, P and gates alone
Saved saved_at(char* base, const Dims& d, bool states);

struct Args {
  Dims d;
  const void *q, *k, *v;            // [B,Hk,T,dk], [B,Hk,T,dk], [B,H,T,dv]
  const float *beta, *log_alpha;    // [B,H,T]
  float scale;
  Saved sv;
  // forward
  const float* S0 = nullptr;        // [B*H][dv][dk] or null (zero)
  void* y = nullptr;                // [B,H,T,dv] or null
  float* ST = nullptr;              // [B*H][dv][dk] or null
  // backward
  const void* dy = nullptr;         // [B,H,T,dv]
  const void* dST = nullptr;        // [B*H][dv][dk] I/O dtype, or null (zero)
  float* E = nullptr;               // scratch [B*H][T][dv]
  float* dS = nullptr;              // scratch [B*H][N][dv][dk]: gradient of chunk-end states
  void *dq = nullptr, *dk_ = nullptr, *dv_ = nullptr;  // like q, k, v
  void *dbeta = nullptr, *dlog_alpha = nullptr;        // [B,H,T] I/O dtype
  void* dS0 = nullptr;              // [B*H][dv][dk] I/O dtype, or null
};

cudaError_t run_fwd(const Args& a, cudaStream_t st);
cudaError_t run_bwd(const Args& a, cudaStream_t st);

}  // namespace ffma
}  // namespace delta
}  // namespace gradlev
