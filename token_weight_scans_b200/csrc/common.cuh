// Shared device/host helpers of the GradLev scan library (CUDA, sm_100a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <atomic>

#include "gradlev.h"

namespace gradlev {

// ---------------------------------------------------------------- dtype I/O
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Device status word at the start of every workspace (see gradlev_device_status).
struct DeviceStatus {
  unsigned int code;    // 0 = ok, else a gradlev_status value
  unsigned int where;   // kernel-specific location of the failed wait
  unsigned int pad[2];
};

// Launch accounting for gradlev_last_launch_count(): every entry point resets the
// count, every kernel launch adds one.
void count_launch();
void reset_launch_count();

// Opts a kernel whose dynamic shared memory depends on the call's sizes into all that the device
// has, once per device (`done`: one bit each, a static of that kernel). The limit belongs to the
// kernel, not to the call: set to a call's own size, another host thread's narrower call could
// lower it again between this call's setting and its launch, which then fails.
inline cudaError_t allow_smem(const void* kernel, std::atomic<uint64_t>& done) {
  int dev = 0, most = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit && (done.load() & bit)) return cudaSuccess;
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             most - (int)fa.sharedSizeBytes);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

}  // namespace gradlev
