// tma_host.cuh -- host-side TMA tensor-map encoding (driver entry point
// looked up through the runtime, so the library needs no libcuda link).
#pragma once

#include <atomic>

#include <cuda.h>
#include <cuda_runtime.h>

namespace gqa {
namespace tma {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t,
                                  void *, const cuuint64_t *, const cuuint64_t *,
                                  const cuuint32_t *, const cuuint32_t *,
                                  CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);

// Looked up until it is found; threads that call for the first time together
// each look, and store the same.
inline EncodeTiledFn encode_fn() {
  static std::atomic<EncodeTiledFn> found{nullptr};
  EncodeTiledFn fn = found.load(std::memory_order_acquire);
  if (fn) return fn;
  void *ptr = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault,
                              &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess) {
    fn = reinterpret_cast<EncodeTiledFn>(ptr);
    found.store(fn, std::memory_order_release);
  } else {
    cudaGetLastError();
  }
  return fn;
}

// bf16 tensor of `heads` x `rows` rows of d elements, boxes of 64 columns x
// box_rows rows x 1, 128-byte swizzle.  A 2-D map when heads == 0.
inline bool make_bf16_map(CUtensorMap *map, const void *base, int d, long long rows,
                          int heads, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t rank = heads > 0 ? 3 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)(heads > 0 ? heads : 1)};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)rows * d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  auto encode = [&] {
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  // The driver's entry points want the device's context current, which the
  // runtime makes it only with a thread's first call that needs one: a thread
  // that has used the device for nothing yet comes here without.  (Allowed in a
  // capture; the device stays the thread's.)
  int dev = 0;
  if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess &&
      cudaSetDevice(dev) == cudaSuccess)
    r = encode();
  return r == CUDA_SUCCESS;
}

}  // namespace tma
}  // namespace gqa
