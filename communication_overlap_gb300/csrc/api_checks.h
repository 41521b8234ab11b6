// Argument checks that the C entry points of the plan-free operators share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "fo.h"

namespace fo {

inline bool type_ok(fo_type t) { return t == FO_TYPE_BF16 || t == FO_TYPE_F32; }

// Sizes that the kernels index with 32-bit rows and columns.
inline bool fits_int32(int64_t n) { return n >= 0 && n <= (int64_t(1) << 31) - 256; }

inline bool device_ok(fo_status* st) {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
    *st = FO_ERR_CUDA;
    return false;
  }
  *st = FO_ERR_UNSUPPORTED;
  return major == 10 && minor == 3;
}

inline bool aligned_type(const void* p, fo_type t) {
  return (reinterpret_cast<uintptr_t>(p) & (t == FO_TYPE_BF16 ? 1u : 3u)) == 0;
}

}  // namespace fo
