// Device helpers of the kernels around the expert layer's products: eight
// elements at a time between memory and fp32, and sums over a warp.
#pragma once

#include <cstdint>
#include <mutex>
#include <type_traits>

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

// Two fp32 values that one instruction takes at once.
struct Pair {
  uint64_t v;
  __device__ __forceinline__ static Pair of(float lo, float hi) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(lo), "f"(hi));
    return p;
  }
  __device__ __forceinline__ static Pair of(float x) { return of(x, x); }
  __device__ __forceinline__ void get(float& lo, float& hi) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
  }
  __device__ __forceinline__ float sum() const {
    float lo, hi;
    get(lo, hi);
    return lo + hi;
  }
};
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}

template <typename T>
__device__ __forceinline__ void pairs_of(const Pack8<T>& p, Pair (&x)[4]) {
  float v[8];
  p.get(v);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = Pair::of(v[2 * i], v[2 * i + 1]);
}

__device__ __forceinline__ void pairs_of(const float (&v)[8], Pair (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = Pair::of(v[2 * i], v[2 * i + 1]);
}

// store8 by a whole warp; `in`: this lane's eights are to be stored.  Of fp32 two lanes
// trade halves, so that a store of theirs is 32 bytes in one piece: half a sector each
// costs twice the traffic to L2.  So the odd lane's eights lie right behind the even
// one's wherever either is to store: where lanes run over rows, an even number of eights
// to a row, or rows that follow each other without a gap.
template <typename T>
__device__ __forceinline__ void store8_warp(T* p, bool in, const float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    if (in) store8(p, v);
  } else {
    const bool odd = threadIdx.x & 1;
    const bool other = __shfl_xor_sync(0xffffffffu, int(in), 1) != 0;
    float4 got;
    got.x = __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[4], 1);
    got.y = __shfl_xor_sync(0xffffffffu, odd ? v[1] : v[5], 1);
    got.z = __shfl_xor_sync(0xffffffffu, odd ? v[2] : v[6], 1);
    got.w = __shfl_xor_sync(0xffffffffu, odd ? v[3] : v[7], 1);
    const float4 lo = make_float4(v[0], v[1], v[2], v[3]), hi = make_float4(v[4], v[5], v[6], v[7]);
    // the even lane's eight, then the odd one's
    if (odd ? other : in) __stcs(reinterpret_cast<float4*>(odd ? p - 4 : p), odd ? got : lo);
    if (odd ? in : other) __stcs(reinterpret_cast<float4*>(odd ? p + 4 : p + 8), odd ? hi : got);
  }
}
template <typename T>
__device__ __forceinline__ void store8_warp(T* p, bool in, const Pair (&x)[4]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i].get(v[2 * i], v[2 * i + 1]);
  store8_warp(p, in, v);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A ring in shared memory that a thread fills for itself, rows ahead of their use: no
// other thread reads its pieces, so no barrier guards them.  Piece i of stage s lies
// at (s * pieces + i) * threads + thread, 16 bytes each.
struct OwnRing {
  uint32_t base;        // of this thread's first piece
  uint32_t step;        // bytes from one piece to the next

  __device__ __forceinline__ OwnRing(const void* smem)
      : base(smem_u32(smem) + threadIdx.x * 16), step(blockDim.x * 16) {}
  __device__ __forceinline__ uint32_t at(int piece) const { return base + uint32_t(piece) * step; }
  // The row's eight elements from `col` on into the ring from piece `piece` on, where they
  // exist (col < limit).  A lane's eight fp32 values are two copies, each of half a
  // sector per lane: through L1, where the second finds what the first brought.  (Past
  // L1 both go to L2, whose tags then bind: 16384 x 4096 in fp32 at 4.7 TB/s.)
  template <typename T>
  __device__ __forceinline__ void fetch(int piece, const T* row, int col, int limit) const {
    if (col >= limit) return;
    if constexpr (sizeof(T) == 2) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at(piece)), "l"(row + col)
                   : "memory");
    } else {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(at(piece)), "l"(row + col)
                   : "memory");
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(at(piece + 1)),
                   "l"(row + col + 4)
                   : "memory");
    }
  }
  template <typename T>
  __device__ __forceinline__ void get(int piece, Pack8<T>& p) const {
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(p.w[i].x), "=r"(p.w[i].y), "=r"(p.w[i].z), "=r"(p.w[i].w)
                   : "r"(at(piece + i))
                   : "memory");
  }
  // eight fp32 values of the thread's own
  __device__ __forceinline__ void put(int piece, const float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at(piece + i)), "f"(v[4 * i]),
                   "f"(v[4 * i + 1]), "f"(v[4 * i + 2]), "f"(v[4 * i + 3])
                   : "memory");
  }
  __device__ __forceinline__ static void commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  template <int N>      // all but the last N groups have arrived
  __device__ __forceinline__ static void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
  }
};

// Eight elements of a ring's pieces as pairs.
template <typename T>
__device__ __forceinline__ void get_pairs(const OwnRing& ring, int piece, Pair (&x)[4]) {
  Pack8<T> p;
  ring.get(piece, p);
  pairs_of(p, x);
}

// E neighbouring elements of a row that need not lie on 16 bytes: two where all rows
// start on two elements and have an even number, else one.
template <typename T, int E>
struct Few {
  static_assert(E == 1 || E == 2, "one element or two");
  using Word = typename std::conditional<sizeof(T) * E == 2, uint16_t,
               typename std::conditional<sizeof(T) * E == 4, uint32_t, uint2>::type>::type;
  Word w;
  __device__ __forceinline__ void zero() {
    if constexpr (sizeof(Word) == 8)
      w = make_uint2(0, 0);
    else
      w = 0;
  }
  __device__ __forceinline__ void load(const T* p) { w = __ldcs(reinterpret_cast<const Word*>(p)); }
  __device__ __forceinline__ void get(float (&v)[E]) const {
    if constexpr (sizeof(Word) == 8) {
      v[0] = __uint_as_float(w.x);
      v[E - 1] = __uint_as_float(w.y);
    } else if constexpr (E == 2) {
      v[0] = bf16lo(w);
      v[E - 1] = bf16hi(w);
    } else if constexpr (sizeof(T) == 4) {
      v[0] = __uint_as_float(w);
    } else {
      v[0] = widen(w);
    }
  }
  __device__ __forceinline__ static void store(T* p, const float (&v)[E]) {
    if constexpr (sizeof(Word) == 8)
      __stcs(reinterpret_cast<uint2*>(p), make_uint2(__float_as_uint(v[0]), __float_as_uint(v[E - 1])));
    else if constexpr (E == 2)
      __stcs(reinterpret_cast<uint32_t*>(p), pack_bf16x2(v[0], v[E - 1]));
    else
      __stcs(p, narrow<T>(v[0]));
  }
};

// Whether rows start on `bytes` bytes.
inline bool rows_on(const void* p, int64_t stride, fo_type type, int bytes) {
  const int64_t size = type == FO_TYPE_BF16 ? 2 : 4;
  return ((reinterpret_cast<uintptr_t>(p) | uintptr_t(stride * size)) & (bytes - 1)) == 0;
}
// And on two elements.
inline bool rows_on_two(const void* p, int64_t stride, fo_type type) {
  return rows_on(p, stride, type, type == FO_TYPE_BF16 ? 4 : 8);
}

// The current device's SMs.
inline fo_status sm_count(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FO_ERR_CUDA;
  return FO_OK;
}

// Lets a kernel take up to kBlockSmem bytes of dynamic shared memory, once per
// kernel and device (not a launch's own size: another thread's launch may follow).
constexpr int kBlockSmem = 220 * 1024;
template <auto K>
fo_status allow_smem() {
  static std::once_flag once[64];
  static cudaError_t err[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FO_ERR_CUDA;
  const int slot = dev < 64 ? dev : 63;
  std::call_once(once[slot], [&] {
    err[slot] = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, kBlockSmem);
  });
  return err[slot] == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace fo
