// host_checks.h — the argument checks the C ABI's translation units share.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "flint_moe.h"

namespace flint {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Required pointer: non-null and 16-byte aligned.
inline bool req(const void* p) { return p != nullptr && aligned16(p); }
// Small fp32 / int32 vectors (offsets, routing outputs): 4-byte alignment.
inline bool req4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool opt4(const void* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + bn && b0 < a0 + an;
}

inline int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

inline flint_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return FLINT_OK;
  (void)cudaGetLastError();  // clear a non-sticky launch error
  return FLINT_ERR_CUDA;
}

}  // namespace flint
