// Entry points of the chunked gated delta rule: argument checks, workspace layout and
// the choice of a kernel family. No device memory is allocated here.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "delta.h"
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
  if ((long long)B * H * T >= (1LL << 31) || (long long)B * H * 16 >= (1LL << 31))
    return GRADLEV_ERR_UNSUPPORTED;
  return GRADLEV_OK;
}

Dims dims(int B, int H, int Hk, int T, int dk, int dv, gradlev_dtype dt) {
  return Dims{B, H, Hk, T, dk, dv, dt == GRADLEV_BF16};
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

size_t ckpt_bytes(const Dims& d) { return ffma::saved_bytes(d, true); }

size_t bwd_scratch(const Dims& d) {  // E and the chunk-end gradients of the state
  return up256(d.BH() * d.T * d.dv * sizeof(float)) +
         up256(d.BH() * ffma::chunks(d.T) * d.dv * d.dk * sizeof(float));
}

size_t ws_bytes_of(const Dims& d, int is_bwd) {
  if (!is_bwd) return kStatusBytes + ffma::saved_bytes(d, false);
  return kStatusBytes + bwd_scratch(d) + ckpt_bytes(d);
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

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
      !aligned(ckpt, 256) || !aligned(workspace, 256))
    return GRADLEV_ERR_INVALID_ARG;
  const Dims d = dims(B, H, Hk, T, d_k, d_v, dt);
  if (ws_bytes < ws_bytes_of(d, 0)) return GRADLEV_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (cudaMemsetAsync(ws, 0, sizeof(DeviceStatus), st) != cudaSuccess) return GRADLEV_ERR_CUDA;
  ffma::Args a{d, q, k, v, beta, log_alpha, scale,
               ckpt ? ffma::saved_at(static_cast<char*>(ckpt), d, true)
                    : ffma::saved_at(ws + kStatusBytes, d, false)};
  a.S0 = S0;
  a.y = y;
  a.ST = ST;
  return ffma::run_fwd(a, st) == cudaSuccess ? GRADLEV_OK : GRADLEV_ERR_CUDA;
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
  char* scratch = ws + kStatusBytes;
  char* saved = ckpt ? static_cast<char*>(const_cast<void*>(ckpt)) : scratch + bwd_scratch(d);
  ffma::Args a{d, q, k, v, beta, log_alpha, scale, ffma::saved_at(saved, d, true)};
  if (!ckpt) {
    a.S0 = S0;
    if (ffma::run_fwd(a, st) != cudaSuccess) return GRADLEV_ERR_CUDA;
  }
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
  return ffma::run_bwd(a, st) == cudaSuccess ? GRADLEV_OK : GRADLEV_ERR_CUDA;
}

}  // extern "C"
