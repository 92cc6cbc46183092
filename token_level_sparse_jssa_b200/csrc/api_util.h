// Host-side helpers shared by the entry points' files (api.cu, api_paged.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "jssa.h"

namespace jssa {

constexpr size_t kAlign = 256;
constexpr int kMaxDevices = 64;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline int num_sms_current() {
  static int cache[kMaxDevices] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
  if (cache[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return -1;
    cache[dev] = n;
  }
  return cache[dev];
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline jssa_status cu(cudaError_t e) {
  if (e == cudaSuccess) return JSSA_OK;
  if (e == cudaErrorNotSupported) return JSSA_ERR_UNSUPPORTED;
  return JSSA_ERR_CUDA;
}

}  // namespace jssa
