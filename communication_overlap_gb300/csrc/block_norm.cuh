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

// E values of a gain or of a gate's row, which need not lie on 16 bytes.
template <int E>
__device__ __forceinline__ void load_few_param(const void* p, int64_t i, bool f32, float (&v)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e)
    v[e] = f32 ? __ldg(static_cast<const float*>(p) + i + e)
               : widen(__ldg(static_cast<const uint16_t*>(p) + i + e));
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

// A token's own row of the gate on its way to the L2, with the token's other rows, as its
// factors are waited for (16384 x 4096 in bf16 with a gate per token 167 -> 141 us, and
// back 266 -> 239).
__device__ __forceinline__ void prefetch_gate(const NormArgs& a, int64_t t, int col) {
  if (a.gate_rows != 1 || a.gate_stride == 0) return;
  const int64_t i = t * a.gate_stride + col;
  const void* p = a.params_f32 ? static_cast<const void*>(static_cast<const float*>(a.gate) + i)
                               : static_cast<const uint16_t*>(a.gate) + i;
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Sums over the warps of a CTA of N values per thread, the same on every thread:
// by shuffles, then through shared memory in warp order.  Every thread of the CTA
// calls it; buf: [2][N][32], the halves taken in turn, so that one barrier per sum
// is enough.
template <int N>
__device__ __forceinline__ void cta_sums(float (&v)[N], float* buf, int& turn) {
  const int warps = int(blockDim.x) >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (warps == 1) return;
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
    for (int w = 0; w < warps; ++w) sum += at[i * 32 + w];
    v[i] = sum;
  }
}

// The threads of a row, one of several of a CTA: they meet at a barrier of their
// own, so that a CTA's rows need not keep step.
struct RowGroup {
  int warps;      // of the row
  int index;      // of the row in the CTA
  int tid;        // of the row's threads

  __device__ __forceinline__ static RowGroup of(int warps) {
    const int index = int(threadIdx.x >> 5) / warps;
    return {warps, index, int(threadIdx.x) - index * warps * 32};
  }
  // cta_sums over the row, of up to 16 warps.  buf, zeros at first: of one value [2][32]
  // (a row's warps take slots from a multiple of four on), of three [2][8 rows][3][16].
  template <int N>
  __device__ __forceinline__ void sums(float (&v)[N], float* buf, int& turn) const {
    const int lane = tid & 31;
    if constexpr (N == 3) {
      // the lanes share the values out on the first two steps: the four quarters of the
      // warp, by their lanes' bits 4 and 3, then add up v0, v1, v2 and nothing
      const bool hi = lane & 16, odd = lane & 8;
      const float give = hi ? v[0] : v[2], keep = hi ? v[2] : v[0];
      const float a = keep + __shfl_xor_sync(0xffffffffu, give, 16);          // v0 or v2
      const float give1 = hi ? v[1] : 0.0f, keep1 = hi ? 0.0f : v[1];
      const float b = keep1 + __shfl_xor_sync(0xffffffffu, give1, 16);        // v1 or 0
      float s = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (warps == 1) {
        v[0] = __shfl_sync(0xffffffffu, s, 0);
        v[1] = __shfl_sync(0xffffffffu, s, 8);
        v[2] = __shfl_sync(0xffffffffu, s, 16);
        return;
      }
      // value i of warp w at i * 16 + w
      float* at = buf + (turn * 8 + index) * 3 * 16;
      turn ^= 1;
      if ((lane & 7) == 0 && lane < 24) at[(lane >> 3) * 16 + (tid >> 5)] = s;
      meet();
      // a quarter of the warp adds a value's sums, two warps' to a lane
      const float2 p = *reinterpret_cast<const float2*>(at + min(lane >> 3, 2) * 16 + (lane & 7) * 2);
      s = p.x + p.y;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      v[0] = __shfl_sync(0xffffffffu, s, 0);
      v[1] = __shfl_sync(0xffffffffu, s, 8);
      v[2] = __shfl_sync(0xffffffffu, s, 16);
    } else {
      static_assert(N == 1, "one value or three");
      v[0] = warp_sum(v[0]);
      if (warps == 1) return;
      float* at = buf + turn * 32 + index * ((warps + 3) & ~3);
      turn ^= 1;
      if (lane == 0) at[tid >> 5] = v[0];
      meet();
      float sum = 0.0f;
      for (int w = 0; w < warps; w += 4) {
        const float4 f = *reinterpret_cast<const float4*>(at + w);
        sum += (f.x + f.y) + (f.z + f.w);
      }
      v[0] = sum;
    }
  }
  __device__ __forceinline__ void meet() const {
    asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(warps * 32) : "memory");
  }
};

// How rows lie over threads: NV times eight columns per thread, and several rows to a
// CTA where one has few warps.
struct RowShape {
  int nv, warps, rows, threads;
};
inline RowShape row_shape(int64_t hidden, int nv, int cta_warps) {
  RowShape s;
  s.nv = nv;
  s.warps = hidden > 0 ? int((hidden + 256 * nv - 1) / (256 * nv)) : 1;
  s.rows = s.warps <= cta_warps ? cta_warps / s.warps : 1;
  s.threads = s.rows * s.warps * 32;
  return s;
}

// scale gate post of E columns (factors that are not given left out).
template <int E>
__device__ __forceinline__ void load_few_factor(const NormArgs& a, int col, int64_t gate_row,
                                                float (&w)[E]) {
  float p[E];
#pragma unroll
  for (int e = 0; e < E; ++e) w[e] = a.scale;
  if (a.gate != nullptr) {
    load_few_param<E>(a.gate, gate_row + col, a.params_f32, p);
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] *= p[e];
  }
  if (a.post != nullptr) {
    load_few_param<E>(a.post, col, a.params_f32, p);
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] *= p[e];
  }
}

// scale gate post of eight columns (factors that are not given left out).
__device__ __forceinline__ void load_factor(const NormArgs& a, int col, int64_t gate_row,
                                            float (&w)[8]) {
  float p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = a.scale;
  if (a.gate != nullptr) {
    load_param<8>(a.gate, gate_row + col, a.params_f32, p);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] *= p[i];
  }
  if (a.post != nullptr) {
    load_param<8>(a.post, col, a.params_f32, p);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] *= p[i];
  }
}

inline bool norm_on_16(const void* p, int64_t stride, int64_t size) {
  return ((reinterpret_cast<uintptr_t>(p) | uintptr_t(stride * size)) & 15) == 0;
}
// Whether all rows of the forward call's tensors start on two elements.
inline bool norm_rows_on_two(const NormArgs& a, fo_type type, fo_type stream_type) {
  return a.hidden % 2 == 0 && rows_on_two(a.x, a.x_stride, type) &&
         rows_on_two(a.residual, a.residual_stride, stream_type) &&
         rows_on_two(a.sum, a.sum_stride, stream_type) && rows_on_two(a.y, a.y_stride, type);
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
