// salr_host.h - host helpers shared by the library's translation units.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/salr.h"

namespace salr {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return SALR_OK;
  return e == cudaErrorMemoryAllocation ? SALR_ERR_OOM : SALR_ERR_CUDA;
}

#define SALR_TRY(expr)                      \
  do {                                      \
    const cudaError_t e_ = (expr);          \
    if (e_ != cudaSuccess) return cuda_status(e_); \
  } while (0)

inline int device_sms(int dev) {
  static std::atomic<int> cache[64];  // zero-initialised: not looked up yet
  if (dev >= 0 && dev < 64 && cache[dev]) return cache[dev];
  int n = 0;
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n > 0 ? n : 1;
}

}  // namespace salr
