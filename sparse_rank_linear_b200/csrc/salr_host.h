// salr_host.h - host helpers shared by the library's translation units.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "../../include/salr.h"

namespace salr {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Span {  // memory of an argument; NULL: not given
  const void* at;
  size_t bytes;
};
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.at && b.at && x < y + b.bytes && y < x + a.bytes;
}
// Whether a written argument (the first `outputs` of `spans`) overlaps another one.
template <size_t N>
bool outputs_overlap(const Span (&spans)[N], size_t outputs) {
  for (size_t i = 0; i < outputs; ++i)
    for (size_t j = i + 1; j < N; ++j)
      if (overlap(spans[i], spans[j])) return true;
  return false;
}

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
