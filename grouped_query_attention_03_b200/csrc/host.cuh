// host.cuh -- host-side helpers shared by the entry points: per-device
// facts, checked size products, pointer alignment, launch errors.
#pragma once

#include <climits>
#include <cstdint>
#include <initializer_list>
#include <mutex>

#include <cuda_runtime.h>

#include "../../include/gqa.h"

namespace gqa {
namespace host {

struct DeviceInfo {
  int sms = 0;
  int major = 0;
  int id = 0;
};

inline gqa_status device_info(DeviceInfo *out) {
  static std::mutex mu;
  static DeviceInfo cache[64];
  static bool have[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (!have[dev]) {
    DeviceInfo d;
    d.id = dev;
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) !=
            cudaSuccess ||
        cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor,
                               dev) != cudaSuccess) {
      cudaGetLastError();
      return GQA_ERR_CUDA;
    }
    cache[dev] = d;
    have[dev] = true;
  }
  *out = cache[dev];
  return out->major == 10 ? GQA_OK : GQA_ERR_DEVICE;
}

// a*b*... in int64 with overflow detection (all factors >= 0).
inline bool mul_ok(int64_t *acc, int64_t f) {
  if (f < 0) return false;
  if (f != 0 && *acc > INT64_MAX / f) return false;
  *acc *= f;
  return true;
}

inline bool elems(int64_t *out, std::initializer_list<int64_t> dims) {
  int64_t acc = 1;
  for (int64_t d : dims)
    if (!mul_ok(&acc, d)) return false;
  *out = acc;
  return true;
}

inline bool aligned16(const void *p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

inline gqa_status check_heads(int Hq, int Hkv, int d) {
  if (Hq <= 0 || Hkv <= 0 || d <= 0) return GQA_ERR_SHAPE;
  if (Hq % Hkv != 0) return GQA_ERR_GROUPS;
  return GQA_OK;
}

inline gqa_status check_window(int window) {
  return (window == 0 || window < -1) ? GQA_ERR_WINDOW : GQA_OK;
}

inline gqa_status launch_status() {
  return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

// Turns a launch call's result into a status, clearing the error.
inline gqa_status launched(cudaError_t e) {
  if (e == cudaSuccess) return GQA_OK;
  cudaGetLastError();
  return GQA_ERR_CUDA;
}

inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// Raise a kernel's dynamic shared memory limit, once per device (the
// attribute belongs to the device's copy of the function).  `done` is the
// instantiation's own table; two threads racing set the same value twice.
template <typename F>
inline gqa_status allow_smem(F *kernel, int bytes, int dev, bool (&done)[64]) {
  if (done[dev]) return GQA_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  done[dev] = true;
  return GQA_OK;
}

}  // namespace host
}  // namespace gqa
