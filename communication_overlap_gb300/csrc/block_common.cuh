// Device helpers of the kernels around the expert layer's products: eight
// elements at a time between memory and fp32, and sums over a warp.
#pragma once

#include <cstdint>

#include "block_internal.h"
#include "device_common.cuh"

namespace fo {

// Elements as they lie in memory: uint16_t for bf16, float.
__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float(uint32_t(x) << 16); }
__device__ __forceinline__ float widen(float x) { return x; }
template <typename T>
__device__ __forceinline__ T narrow(float x) {
  if constexpr (sizeof(T) == 2) {
    const __nv_bfloat16 h = __float2bfloat16_rn(x);
    return *reinterpret_cast<const uint16_t*>(&h);
  } else {
    return x;
  }
}

// Eight consecutive elements, still packed; p on 16 bytes.
template <typename T>
struct Pack8 {
  uint4 w[sizeof(T) / 2];

  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  // data that nothing reads again soon
  __device__ __forceinline__ void load_once(const T* p) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (sizeof(T) == 2) {
      v[0] = bf16lo(w[0].x), v[1] = bf16hi(w[0].x), v[2] = bf16lo(w[0].y), v[3] = bf16hi(w[0].y);
      v[4] = bf16lo(w[0].z), v[5] = bf16hi(w[0].z), v[6] = bf16lo(w[0].w), v[7] = bf16hi(w[0].w);
    } else {
      v[0] = __uint_as_float(w[0].x), v[1] = __uint_as_float(w[0].y);
      v[2] = __uint_as_float(w[0].z), v[3] = __uint_as_float(w[0].w);
      v[4] = __uint_as_float(w[1].x), v[5] = __uint_as_float(w[1].y);
      v[6] = __uint_as_float(w[1].z), v[7] = __uint_as_float(w[1].w);
    }
  }
};

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    __stcs(reinterpret_cast<uint4*>(p),
           make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7])));
  } else {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

}  // namespace fo
