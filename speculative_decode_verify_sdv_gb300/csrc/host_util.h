// Host-side helpers of the entry points outside api.cu.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "sdv.h"

namespace sdv {

constexpr size_t kHeaderBytes = 256;  // a workspace's head: word 0 is the status; zero between calls

inline bool is_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline sdv_status status_of(cudaError_t e) { return e == cudaSuccess ? SDV_OK : SDV_ERR_CUDA; }

inline int attribute_of_device(cudaDeviceAttr attr) {
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&v, attr, dev) != cudaSuccess) return 0;
  return v;
}

inline int sm_count() { return attribute_of_device(cudaDevAttrMultiProcessorCount); }

inline size_t round_256(size_t b) { return (b + 255) / 256 * 256; }

}  // namespace sdv
