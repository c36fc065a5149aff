// Entry points of the chunked gated delta rule: argument checks, workspace layout and
// the choice of a kernel family. No device memory is allocated here.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "delta.h"
#include "delta_tc.h"
#include "dispatch.h"
#include "gradlev.h"

namespace gradlev {
namespace delta {
namespace {

gradlev_status check_shape(int B, int H, int Hk, int T, int dk, int dv, gradlev_dtype dt) {
  if (B <= 0 || H <= 0 || Hk <= 0 || T <= 0 || dk <= 0 || dv <= 0) return GRADLEV_ERR_INVALID_ARG;
  if (dt != GRADLEV_F32 && dt != GRADLEV_BF16) return GRADLEV_ERR_INVALID_ARG;
  if (H % Hk != 0) return GRADLEV_ERR_UNSUPPORTED;
  if (dk % 8 != 0 || dv % 8 != 0 || dk > 256 || dv > 256) return GRADLEV_ERR_UNSUPPORTED;
  const long long BH = (long long)B * H;  // B*H*T itself may pass 64 bits
  if (BH >= 1LL << 27 || BH * T >= 1LL << 31) return GRADLEV_ERR_UNSUPPORTED;
  return GRADLEV_OK;
}

Dims dims(int B, int H, int Hk, int T, int dk, int dv, gradlev_dtype dt) {
  return Dims{B, H, Hk, T, dk, dv, dt == GRADLEV_BF16};
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// bf16 calls take the tensor cores from W = B H T d_k d_v > 2^24 on, and where few long scans are
// walked in segments. Below, their latency and their padding to 128 columns cost more than the
// float32 kernels, which are also the more exact ones (1.7e-3 off, the outputs' own rounding; the
// tensor cores' 1.7 to 2.4e-3 over many gates, but single gates whose gradient happens to be small up
// to 3e-2). Kernels of the forward with the last state: H16 T1 d128 13 against 28 us, T64 (2^24) 16
// against 27, T256 31 against 40, T1000 97 against 85; of forward and gradients: d128 H16 T64 63
// against 42 us, H1 T1024 214 against 171 (both 2^24), d64 B4 H8 T256 (2^25) 66 against 68, d48 B4 H8
// T256 (2^24) 58 against 69. H2 T8192 d24, in segments, 347 against 244 and 768 against 438 us.
bool use_tc(const Dims& d) {
  return tc::shape_ok(d) &&
         (d.BH() * d.T * d.dk * d.dv > (1u << 24) || tc::seg_plan(d).nseg > 1);
}

size_t ckpt_bytes(const Dims& d) {
  return use_tc(d) ? tc::saved_bytes(d) : ffma::saved_bytes(d, true);
}

size_t fwd_scratch(const Dims& d) {
  return use_tc(d) ? tc::fwd_scratch_bytes(d) : ffma::saved_bytes(d, false);
}

size_t bwd_scratch(const Dims& d) {  // E and the chunk-end gradients of the state
  if (use_tc(d)) return tc::bwd_scratch_bytes(d);
  return up256(d.BH() * d.T * d.dv * sizeof(float)) +
         up256(d.BH() * ffma::chunks(d.T) * d.dv * d.dk * sizeof(float));
}

// The backward without checkpoints runs the forward into its own workspace. The forward's
// scratch is dead by the time the backward's is written, so the two share their place.
size_t ws_bytes_of(const Dims& d, int is_bwd) {
  if (!is_bwd) return kStatusBytes + fwd_scratch(d);
  const size_t f = fwd_scratch(d), b = bwd_scratch(d);
  return kStatusBytes + (f > b ? f : b) + ckpt_bytes(d);
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

// The forward with its scratch behind the status word of `ws`; saved: the checkpoints, or
// null; y: null for the checkpoints alone.
cudaError_t fwd_run(const Dims& d, const void* q, const void* k, const void* v, const float* beta,
                    const float* log_alpha, float scale, const float* S0, void* y, float* ST,
                    char* saved, char* ws, cudaStream_t st) {
  if (use_tc(d)) {
    tc::Args a{d, q, k, v, beta, log_alpha, scale, reinterpret_cast<DeviceStatus*>(ws),
               kWaitTimeoutNs, tc::mats_at(ws + kStatusBytes, d, saved != nullptr)};
    if (saved) {
      a.sv = tc::saved_at(saved, d);
      a.m.Kw = a.sv.Kw;
      a.m.Wq = a.sv.Wq;
      a.m.Wq2 = a.sv.Wq2;
      a.m.Pv = a.sv.Pv;
      a.m.gates = a.sv.gates;
    }
    a.S0 = S0;
    a.y = y;
    a.ST = ST;
    a.inject = take_inject(INJ_DELTA_FWD, 1, &a.timeout_ns);
    tc::set_segments(a, ws + kStatusBytes + tc::fwd_scratch_bytes(d) - tc::seg_bytes(d, true), a.sv.M);
    return tc::run_fwd(a, st);
  }
  ffma::Args a{d, q, k, v, beta, log_alpha, scale,
               saved ? ffma::saved_at(saved, d, true) : ffma::saved_at(ws + kStatusBytes, d, false)};
  a.S0 = S0;
  a.y = y;
  a.ST = ST;
  return ffma::run_fwd(a, st);
}

}  // namespace
}  // namespace delta
}  // namespace gradlev

using namespace gradlev;
using namespace gradlev::delta;

extern "C" {

gradlev_status gradlev_delta_supported(int B, int H, int Hk, int T, int d_k, int d_v,
                                       gradlev_dtype dt) {
  return check_shape(B, H, Hk, T, d_k, d_v, dt);
}

size_t gradlev_delta_workspace_bytes(int B, int H, int Hk, int T, int d_k, int d_v,
                                     gradlev_dtype dt, int is_bwd) {
  if (check_shape(B, H, Hk, T, d_k, d_v, dt) != GRADLEV_OK) return 0;
  return ws_bytes_of(dims(B, H, Hk, T, d_k, d_v, dt), is_bwd);
}

size_t gradlev_delta_ckpt_bytes(int B, int H, int Hk, int T, int d_k, int d_v, gradlev_dtype dt) {
  if (check_shape(B, H, Hk, T, d_k, d_v, dt) != GRADLEV_OK) return 0;
  return ckpt_bytes(dims(B, H, Hk, T, d_k, d_v, dt));
}

gradlev_status gradlev_delta_fwd(int B, int H, int Hk, int T, int d_k, int d_v, gradlev_dtype dt,
                                 const void* q, const void* k, const void* v, const float* beta,
                                 const float* log_alpha, float scale, const float* S0, void* y,
                                 float* ST, void* ckpt, void* workspace, size_t ws_bytes,
                                 void* stream) {
  reset_launch_count();
  const gradlev_status s = check_shape(B, H, Hk, T, d_k, d_v, dt);
  if (s != GRADLEV_OK) return s;
  if (!q || !k || !v || !beta || !log_alpha || !y || !workspace) return GRADLEV_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(y, 16) ||
      !aligned(beta, 4) || !aligned(log_alpha, 4) || !aligned(S0, 16) || !aligned(ST, 16) ||
      !aligned(ckpt, 256) || !aligned(workspace, 256) || (ST && ST == S0))
    return GRADLEV_ERR_INVALID_ARG;
  const Dims d = dims(B, H, Hk, T, d_k, d_v, dt);
  if (ws_bytes < ws_bytes_of(d, 0)) return GRADLEV_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (cudaMemsetAsync(ws, 0, sizeof(DeviceStatus), st) != cudaSuccess) return GRADLEV_ERR_CUDA;
  return fwd_run(d, q, k, v, beta, log_alpha, scale, S0, y, ST, static_cast<char*>(ckpt), ws, st) ==
                 cudaSuccess
             ? GRADLEV_OK
             : GRADLEV_ERR_CUDA;
}

gradlev_status gradlev_delta_bwd(int B, int H, int Hk, int T, int d_k, int d_v, gradlev_dtype dt,
                                 const void* q, const void* k, const void* v, const float* beta,
                                 const float* log_alpha, float scale, const float* S0,
                                 const void* dy, const void* dST, void* dq, void* dk, void* dv,
                                 void* dbeta, void* dlog_alpha, void* dS0, const void* ckpt,
                                 void* workspace, size_t ws_bytes, void* stream) {
  reset_launch_count();
  const gradlev_status s = check_shape(B, H, Hk, T, d_k, d_v, dt);
  if (s != GRADLEV_OK) return s;
  if (!q || !k || !v || !beta || !log_alpha || !dy || !dq || !dk || !dv || !dbeta || !dlog_alpha ||
      !workspace)
    return GRADLEV_ERR_INVALID_ARG;
  for (const void* p : {q, k, v, dy, dST, (const void*)S0, (const void*)dq, (const void*)dk,
                        (const void*)dv, (const void*)dS0})
    if (!aligned(p, 16)) return GRADLEV_ERR_INVALID_ARG;
  if (!aligned(beta, 4) || !aligned(log_alpha, 4) || !aligned(dbeta, 4) ||
      !aligned(dlog_alpha, 4) || !aligned(ckpt, 256) || !aligned(workspace, 256))
    return GRADLEV_ERR_INVALID_ARG;
  const Dims d = dims(B, H, Hk, T, d_k, d_v, dt);
  if (ws_bytes < ws_bytes_of(d, 1)) return GRADLEV_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (cudaMemsetAsync(ws, 0, sizeof(DeviceStatus), st) != cudaSuccess) return GRADLEV_ERR_CUDA;
  char* saved = static_cast<char*>(const_cast<void*>(ckpt));
  if (!ckpt) {
    const size_t f = fwd_scratch(d), b = bwd_scratch(d);
    saved = ws + kStatusBytes + (f > b ? f : b);
    if (fwd_run(d, q, k, v, beta, log_alpha, scale, S0, nullptr, nullptr, saved, ws, st) != cudaSuccess)
      return GRADLEV_ERR_CUDA;
  }
  char* scratch = ws + kStatusBytes;
  if (use_tc(d)) {
    delta::tc::Args a{d, q, k, v, beta, log_alpha, scale, reinterpret_cast<DeviceStatus*>(ws),
               kWaitTimeoutNs};
    a.sv = delta::tc::saved_at(saved, d);
    a.m.Kw = a.sv.Kw;
    a.m.Wq = a.sv.Wq;
    a.m.Wq2 = a.sv.Wq2;
    a.m.Pv = a.sv.Pv;
    a.m.gates = a.sv.gates;
    a.dy = dy;
    a.dST = dST;
    a.E = reinterpret_cast<delta::tc::bf16*>(scratch);
    a.dS = reinterpret_cast<delta::tc::bf16*>(scratch + delta::tc::token_rows_bytes(d));
    a.dq = dq;
    a.dk_ = dk;
    a.dv_ = dv;
    a.dbeta = dbeta;
    a.dlog_alpha = dlog_alpha;
    a.dS0 = dS0;
    a.inject = take_inject(INJ_DELTA_BWD, 1, &a.timeout_ns);
    delta::tc::set_segments(a, scratch + delta::tc::bwd_scratch_bytes(d) - delta::tc::seg_bytes(d, false),
                            a.sv.M);
    return delta::tc::run_bwd(a, st) == cudaSuccess ? GRADLEV_OK : GRADLEV_ERR_CUDA;
  }
  delta::ffma::Args a{d, q, k, v, beta, log_alpha, scale, delta::ffma::saved_at(saved, d, true)};
  a.dy = dy;
  a.dST = dST;
  a.E = reinterpret_cast<float*>(scratch);
  a.dS = reinterpret_cast<float*>(scratch + up256(d.BH() * T * d_v * sizeof(float)));
  a.dq = dq;
  a.dk_ = dk;
  a.dv_ = dv;
  a.dbeta = dbeta;
  a.dlog_alpha = dlog_alpha;
  a.dS0 = dS0;
  return delta::ffma::run_bwd(a, st) == cudaSuccess ? GRADLEV_OK : GRADLEV_ERR_CUDA;
}

}  // extern "C"
