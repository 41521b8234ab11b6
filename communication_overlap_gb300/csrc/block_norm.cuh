// What the norm's forward and backward kernels share: pieces of a row, its
// parameters, sums over a row's threads.
#pragma once

#include <cstdint>

#include "block_common.cuh"

namespace fo {

// W consecutive elements of a row: eight, on 16 bytes, or one.
template <typename T, int W>
struct Piece {
  static_assert(W == 8 || W == 1, "eight elements or one");
  Pack8<T> p;
  __device__ __forceinline__ void load(const T* at, bool live) {
    if (live)
      p.load_once(at);
    else
      p.zero();
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { p.get(v); }
};
template <typename T>
struct Piece<T, 1> {
  T e;
  __device__ __forceinline__ void load(const T* at, bool live) { e = live ? __ldcs(at) : T(0); }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = widen(e); }
};

template <int W, typename T>
__device__ __forceinline__ void store_piece(T* at, const float (&v)[W]) {
  if constexpr (W == 8)
    store8(at, v);
  else
    __stcs(at, narrow<T>(v[0]));
}

// W values of a gain or of a gate's row, from element i on (bf16 or fp32).
template <int W>
__device__ __forceinline__ void load_param(const void* p, int64_t i, bool f32, float (&v)[W]) {
  if constexpr (W == 1) {
    v[0] = f32 ? __ldg(static_cast<const float*>(p) + i)
               : widen(__ldg(static_cast<const uint16_t*>(p) + i));
  } else if (f32) {
    Pack8<float> q;
    q.load(static_cast<const float*>(p) + i);
    q.get(v);
  } else {
    Pack8<uint16_t> q;
    q.load(static_cast<const uint16_t*>(p) + i);
    q.get(v);
  }
}

// Sums over the row's warps of N values per thread, the same on every thread:
// by shuffles, then through shared memory in warp order.  Every thread of the
// CTA calls it; buf: [2][N][32], the halves taken in turn, so that one barrier
// per sum is enough.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int first_warp, int warps, float* buf,
                                         int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (warps == 1) return;      // (the same for all of the CTA)
  float* at = buf + turn * N * 32;
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) at[i * 32 + (threadIdx.x >> 5)] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float sum = 0.0f;
    for (int w = 0; w < warps; ++w) sum += at[i * 32 + first_warp + w];
    v[i] = sum;
  }
}

inline bool norm_on_16(const void* p, int64_t stride, int64_t size) {
  return ((reinterpret_cast<uintptr_t>(p) | uintptr_t(stride * size)) & 15) == 0;
}
inline int64_t size_of(fo_type t) { return t == FO_TYPE_BF16 ? 2 : 4; }

// Whether all rows of the forward call's tensors lie on 16 bytes.
inline bool norm_rows_on_16(const NormArgs& a, fo_type type, fo_type stream_type) {
  const int64_t p = a.params_f32 ? 4 : 2, x = size_of(type), s = size_of(stream_type);
  return a.hidden % 8 == 0 && norm_on_16(a.x, a.x_stride, x) &&
         norm_on_16(a.residual, a.residual_stride, s) && norm_on_16(a.gate, a.gate_stride, p) &&
         norm_on_16(a.post, 0, p) && norm_on_16(a.pre, 0, p) &&
         norm_on_16(a.sum, a.sum_stride, s) && norm_on_16(a.y, a.y_stride, x);
}

}  // namespace fo
