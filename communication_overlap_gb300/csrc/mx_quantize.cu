// Conversion to and from the microscaled 4-bit form.
//
// Per block of 32 values x_i of a row, with a = max |x_i|:
//   s = 2^(floor(log2 a) - 2),  q_i = the E2M1 value nearest x_i / s.
// floor(log2 a) is a's exponent field and s a power of two, so s and x_i / s
// are exact and the only rounding is the one to E2M1.
//
// Both directions move each byte once and compute almost nothing: HBM bounds
// them, and the instructions per value come close (12 to quantize, 9 back: the
// issue slots are 70% busy).  A CTA takes one block of scales (128 rows x 128
// columns): 256 threads, each 8 rows 16 apart x 8 columns, all loads issued
// before the first use (16 bytes x 8 per thread of bf16), four neighbouring lanes
// to a block of 32.  (512 threads over two blocks of columns, for longer pieces
// of a row: 78 us instead of 53.)
//
// Measured at 32768 x 4096 (bf16, fp32): quantize 53 us (6.4 TB/s) and 89 (6.9),
// gathered rows 56 and 93, transposed 60 (5.7) and 122 (5.0), back 53 (6.4) and
// 91 (6.7).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "moe_internal.h"
#include "mx_common.cuh"

namespace fo {

namespace {

constexpr int kThreads = 256;

// Eight consecutive elements as they are kept.
template <typename T>
struct Eight {
  static constexpr int kWords = 2 * int(sizeof(T));
  uint32_t w[kWords];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // ALIGN: bytes that p is a multiple of, 16, or down to an element
  template <int ALIGN>
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (ALIGN == 16) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else if constexpr (ALIGN == 8) {
#pragma unroll
      for (int i = 0; i < kWords / 2; ++i) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p) + i);
        w[2 * i] = v.x, w[2 * i + 1] = v.y;
      }
    } else if constexpr (ALIGN == 4) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
    } else {      // p + 1 is a multiple of 4 bytes, or p is
      uint32_t h[2] = {p[0], p[7]}, m[3];
      if (reinterpret_cast<uintptr_t>(p) & 2) {
#pragma unroll
        for (int i = 0; i < 3; ++i) m[i] = __ldg(reinterpret_cast<const uint32_t*>(p + 1) + i);
        w[0] = h[0] | m[0] << 16;
        w[1] = __funnelshift_r(m[0], m[1], 16);
        w[2] = __funnelshift_r(m[1], m[2], 16);
        w[3] = m[2] >> 16 | h[1] << 16;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
      }
    }
  }
  __device__ __forceinline__ void load_some(const T* p, int valid) {   // the first of them
    zero();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) {
        if constexpr (sizeof(T) == 2)
          w[i / 2] |= uint32_t(p[i]) << (16 * (i & 1));
        else
          w[i] = __float_as_uint(p[i]);
      }
  }
  // The largest magnitude's fp32 bits.
  __device__ __forceinline__ uint32_t amax() const {
    if constexpr (sizeof(T) == 2) {
      uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
      for (int i = 1; i < 4; ++i)
        asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
      return max(m << 16, m & 0xffff0000u);
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
      return m;
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (sizeof(T) == 2)
      return i & 1 ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]);
    else
      return __uint_as_float(w[i]);
  }
};

struct QuantArgs {
  const void* src;
  int64_t batch_stride, row_stride;
  int64_t rows, cols;
  const int32_t* row_index;
  int64_t src_rows;
  uint8_t* codes;
  uint8_t* scales;
  int32_t row_blocks, col_blocks;
};

// What all rows of all matrices start at a multiple of: 16 bytes, 8, 4 or 2.
int rows_align(const void* p, int64_t batch, int64_t batch_stride, int64_t row_stride,
               int64_t size) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p) | uintptr_t(row_stride * size) |
                         uintptr_t(batch > 1 ? batch_stride * size : 0) | 16;
  return int(bits & (~bits + 1));
}

// Rows of the source (or gathered rows of it) become rows of the result.
// ALIGN: what the rows' addresses are a multiple of, in bytes.
template <typename T, int ALIGN, bool GATHER>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 5 : 3) quantize_rows_kernel(const QuantArgs a) {
  __shared__ __align__(16) uint32_t scale_block[kMxScaleBytes / 4];
  int64_t id = blockIdx.x;
  const int cb = int(id % a.col_blocks);
  id /= a.col_blocks;
  const int rb = int(id % a.row_blocks);
  const int64_t b = id / a.row_blocks;
  const T* src = static_cast<const T*>(a.src) + b * a.batch_stride;
  const int col = (threadIdx.x & 15) * 8;          // of the block's 128
  const int64_t c0 = int64_t(cb) * kMxCols + col;
  const int64_t left = a.cols - c0;
  const int valid = left < 0 ? 0 : (left < 8 ? int(left) : 8);
  const int r0 = threadIdx.x >> 4;                 // 16 rows per pass
  const int64_t pitch = int64_t(a.col_blocks) * 64;
  uint8_t* codes = a.codes + (b * a.row_blocks + rb) * int64_t(kMxRows) * pitch + c0 / 2;
  // which rows, then all loads, then the rest: no load waits for another
  const int64_t first = int64_t(rb) * kMxRows + r0;
  Eight<T> v[8];
  const auto load = [&](int p, const T* from, bool live) {
    if (valid == 8) {
      v[p].zero();
      if (live) v[p].template load<ALIGN>(from);
    } else {
      v[p].load_some(from, live ? valid : 0);
    }
  };
  if constexpr (GATHER) {
    int32_t row[8];                                // -1: a row of zeros
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      row[p] = first + p * 16 < a.rows ? __ldg(a.row_index + first + p * 16) : -1;
      if (row[p] >= a.src_rows) row[p] = -1;
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) load(p, src + int64_t(row[p]) * a.row_stride + c0, row[p] >= 0);
  } else {
    const int left = int(min(a.rows - first, int64_t(kMxRows)));
    const T* from = src + first * a.row_stride + c0;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      load(p, from, p * 16 < left);
      from += 16 * a.row_stride;
    }
  }
  uint8_t* to = codes + int64_t(r0) * pitch;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int r = p * 16 + r0;
    uint32_t m = v[p].amax();
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t s = mx_scale_byte(m);
    const float inv = mx_inverse_scale(s);
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = v[p].value(i) * inv;
    const uint32_t q = mx_encode8(u);
    __stcs(reinterpret_cast<uint32_t*>(to), s == 255u ? 0u : q);
    to += 16 * pitch;
    if ((threadIdx.x & 3) == 0)
      reinterpret_cast<uint8_t*>(scale_block)[mx_scale_row(r) + (col >> 5)] = uint8_t(s);
  }
  __syncthreads();
  if (threadIdx.x < kMxScaleBytes / 4)
    reinterpret_cast<uint32_t*>(a.scales +
                                ((b * a.row_blocks + rb) * a.col_blocks + cb) *
                                    int64_t(kMxScaleBytes))[threadIdx.x] = scale_block[threadIdx.x];
}

// Rows that do not start at 16 bytes are written through shared memory, half a
// block at a time: a warp stores a row in whole words, whatever the row's
// address, and the elements at its ends alone.  (Element by element from
// registers 8190 x 4100 bf16 took 98 us, this way 27.  For reading, where L1
// holds what neighbours share, the same detour took 60 us instead of 23.)
template <typename T>
struct Staged {
  static constexpr int kRows = 64;
  static constexpr int kPitch = kMxCols + 16 / int(sizeof(T));   // elements
  T tile[kRows * kPitch];

  __device__ __forceinline__ T* row(int i) { return tile + i * kPitch; }
  // Row i's first n elements to p; by a warp.
  __device__ __forceinline__ void store(int i, T* p, int n) {
    const int lane = threadIdx.x & 31;
    const T* from = row(i);
    if constexpr (sizeof(T) == 2) {
      const int odd = n > 0 ? int(reinterpret_cast<uintptr_t>(p) >> 1) & 1 : 0;
      const int words = (n - odd) / 2;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = j * 32 + lane;
        if (k < words)
          __stcs(reinterpret_cast<uint32_t*>(p + odd) + k,
                 uint32_t(from[odd + 2 * k]) | uint32_t(from[odd + 2 * k + 1]) << 16);
      }
      if (lane == 0 && odd) p[0] = from[0];
      if (lane == 1 && ((n - odd) & 1)) p[n - 1] = from[n - 1];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j * 32 + lane < n) __stcs(p + j * 32 + lane, from[j * 32 + lane]);
    }
  }
};

// Columns of the source become rows of the result: the tile goes through
// shared memory as [column of the result][row], two rows to a thread, four
// neighbouring lanes to the four blocks of a row pair so that they store 64
// contiguous bytes.  The tile's rows are 128 elements + a shift of 8 words per
// block of 32, which keeps those four lanes' reads in different banks.
template <typename T>
struct TileOf {
  static constexpr int kPitch = kMxRows * int(sizeof(T));      // bytes of a column's 128 rows
  static constexpr int kShift = 8 * 4 * (int(sizeof(T)) / 2);  // bytes per block of 32
  static constexpr int kBytes = kMxCols * kPitch + 4 * kShift;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_cols_kernel(const QuantArgs a) {
  using C = TileOf<T>;
  extern __shared__ __align__(16) uint8_t tile[];
  __shared__ __align__(16) uint32_t scale_block[kMxScaleBytes / 4];
  int64_t id = blockIdx.x;
  const int rb = int(id % a.row_blocks);           // neighbours read neighbouring source columns
  id /= a.row_blocks;
  const int cb = int(id % a.col_blocks);
  const int64_t b = id / a.col_blocks;
  const T* src = static_cast<const T*>(a.src) + b * a.batch_stride;
  const bool vec = ((reinterpret_cast<uintptr_t>(src) |
                     uintptr_t(a.row_stride) * sizeof(T)) & 15) == 0;
  {
    constexpr int kVec = 16 / int(sizeof(T));       // elements of a 16-byte piece
    constexpr int kPieces = kMxRows / kVec;         // pieces of a column
    constexpr int kPer = kMxCols * kPieces / kThreads;
    uint4 w[kPer];
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int i = p * kThreads + threadIdx.x;
      const int c = i / kPieces, r = (i % kPieces) * kVec;
      const int64_t gc = int64_t(cb) * kMxCols + c, gr = int64_t(rb) * kMxRows + r;
      const T* from = src + gc * a.row_stride + gr;
      w[p] = make_uint4(0, 0, 0, 0);
      if (gc < a.cols) {
        if (vec && gr + kVec <= a.rows) {
          w[p] = __ldcs(reinterpret_cast<const uint4*>(from));
        } else {
          T e[kVec];
#pragma unroll
          for (int j = 0; j < kVec; ++j) e[j] = gr + j < a.rows ? from[j] : T(0);
          if constexpr (sizeof(T) == 2) {
            w[p] = make_uint4(e[0] | uint32_t(e[1]) << 16, e[2] | uint32_t(e[3]) << 16,
                              e[4] | uint32_t(e[5]) << 16, e[6] | uint32_t(e[7]) << 16);
          } else {
            w[p] = make_uint4(__float_as_uint(e[0]), __float_as_uint(e[1]),
                              __float_as_uint(e[2]), __float_as_uint(e[3]));
          }
        }
      }
    }
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int i = p * kThreads + threadIdx.x;
      const int c = i / kPieces, r = (i % kPieces) * kVec;
      *reinterpret_cast<uint4*>(tile + c * C::kPitch + (c >> 5) * C::kShift + r * int(sizeof(T))) =
          w[p];
    }
  }
  __syncthreads();
  const int blk = threadIdx.x & 3, r = (threadIdx.x >> 2) * 2;   // rows r and r + 1
  const uint8_t* from = tile + blk * (32 * C::kPitch + C::kShift) + r * int(sizeof(T));
  // both rows' 32 values: a word of two bf16 each, or two words
  constexpr int kW = int(sizeof(T)) / 2;
  uint32_t w[32 * kW];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if constexpr (sizeof(T) == 2) {
      w[i] = *reinterpret_cast<const uint32_t*>(from + i * C::kPitch);
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(from + i * C::kPitch);
      w[2 * i] = v.x, w[2 * i + 1] = v.y;
    }
  }
  uint32_t m0 = 0, m1 = 0;
  if constexpr (sizeof(T) == 2) {
    uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 32; ++i)
      asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
    m0 = m << 16, m1 = m & 0xffff0000u;
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      m0 = max(m0, w[2 * i] & 0x7fffffffu);
      m1 = max(m1, w[2 * i + 1] & 0x7fffffffu);
    }
  }
  const uint32_t s0 = mx_scale_byte(m0), s1 = mx_scale_byte(m1);
  const float i0 = mx_inverse_scale(s0), i1 = mx_inverse_scale(s1);
  uint32_t q0[4], q1[4];
#pragma unroll
  for (int o = 0; o < 4; ++o) {
    float u0[8], u1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = o * 8 + i;
      if constexpr (sizeof(T) == 2) {
        u0[i] = bf16lo(w[at]) * i0, u1[i] = bf16hi(w[at]) * i1;
      } else {
        u0[i] = __uint_as_float(w[2 * at]) * i0, u1[i] = __uint_as_float(w[2 * at + 1]) * i1;
      }
    }
    q0[o] = s0 == 255u ? 0u : mx_encode8(u0);
    q1[o] = s1 == 255u ? 0u : mx_encode8(u1);
  }
  const int64_t pitch = int64_t(a.col_blocks) * 64;
  uint8_t* dst = a.codes + ((b * a.row_blocks + rb) * int64_t(kMxRows) + r) * pitch +
                 int64_t(cb) * 64 + blk * 16;
  __stcs(reinterpret_cast<uint4*>(dst), make_uint4(q0[0], q0[1], q0[2], q0[3]));
  __stcs(reinterpret_cast<uint4*>(dst + pitch), make_uint4(q1[0], q1[1], q1[2], q1[3]));
  uint8_t* sb = reinterpret_cast<uint8_t*>(scale_block);
  sb[mx_scale_row(r) + blk] = uint8_t(s0);
  sb[mx_scale_row(r + 1) + blk] = uint8_t(s1);
  __syncthreads();
  if (threadIdx.x < kMxScaleBytes / 4)
    reinterpret_cast<uint32_t*>(a.scales +
                                ((b * a.row_blocks + rb) * a.col_blocks + cb) *
                                    int64_t(kMxScaleBytes))[threadIdx.x] = scale_block[threadIdx.x];
}

struct DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  void* dst;
  int64_t batch_stride, row_stride;
  int64_t rows, cols;
  int32_t row_blocks, col_blocks;
};

template <typename T, bool STAGED>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const DequantArgs a) {
  int64_t id = blockIdx.x;
  const int cb = int(id % a.col_blocks);
  id /= a.col_blocks;
  const int rb = int(id % a.row_blocks);
  const int64_t b = id / a.row_blocks;
  T* dst = static_cast<T*>(a.dst) + b * a.batch_stride;
  const int col = (threadIdx.x & 15) * 8;
  const int64_t c0 = int64_t(cb) * kMxCols + col;
  const int64_t left = a.cols - c0;
  const int valid = left < 0 ? 0 : (left < 8 ? int(left) : 8);
  const int r0 = threadIdx.x >> 4;
  const int64_t pitch = int64_t(a.col_blocks) * 64;
  const uint8_t* codes = a.codes + (b * a.row_blocks + rb) * int64_t(kMxRows) * pitch + c0 / 2;
  const uint8_t* scales = a.scales + ((b * a.row_blocks + rb) * a.col_blocks + cb) *
                                         int64_t(kMxScaleBytes) + (col >> 5);
  uint32_t q[8];
  uint32_t s[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int r = p * 16 + r0;
    q[p] = __ldcs(reinterpret_cast<const uint32_t*>(codes + r * pitch));
    s[p] = scales[mx_scale_row(r)];
  }
  // whether all of the warp's columns exist
  const bool pair = !STAGED && __all_sync(0xffffffffu, valid == 8);
  // eight values of pass p to `to` (of shared memory where STAGED), if live;
  // by whole warps
  const auto put = [&](int p, T* to, bool live) {
    uint32_t h[4];
    mx_decode8(q[p], h);
    const float scale = mx_scale_value(s[p]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      v[2 * i] = f.x * scale;
      v[2 * i + 1] = f.y * scale;
    }
    if constexpr (sizeof(T) == 2) {
      const uint4 w = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      if (STAGED) {
        *reinterpret_cast<uint4*>(to) = w;
      } else if (live && valid == 8) {
        __stcs(reinterpret_cast<uint4*>(to), w);
      } else if (live) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < valid) to[i] = uint16_t(u[i / 2] >> (16 * (i & 1)));
      }
    } else {
      float4 lo = make_float4(v[0], v[1], v[2], v[3]), hi = make_float4(v[4], v[5], v[6], v[7]);
      if (STAGED) {
        reinterpret_cast<float4*>(to)[0] = lo;
        reinterpret_cast<float4*>(to)[1] = hi;
      } else if (pair) {
        // two neighbouring lanes trade halves, so that each store of theirs is 32
        // bytes in one piece (127 -> 100 us at 32768 x 4096)
        const bool odd = threadIdx.x & 1;
        const float4 give = odd ? lo : hi;
        float4 got;
        got.x = __shfl_xor_sync(0xffffffffu, give.x, 1);
        got.y = __shfl_xor_sync(0xffffffffu, give.y, 1);
        got.z = __shfl_xor_sync(0xffffffffu, give.z, 1);
        got.w = __shfl_xor_sync(0xffffffffu, give.w, 1);
        T* at = odd ? to - 4 : to;
        if (live) {
          __stcs(reinterpret_cast<float4*>(at), odd ? got : lo);
          __stcs(reinterpret_cast<float4*>(at + 8), odd ? hi : got);
        }
      } else if (live) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < valid) to[i] = v[i];
      }
    }
  };
  if constexpr (STAGED) {
    __shared__ __align__(16) Staged<T> staged;
    const int warp = threadIdx.x >> 5;
    const int n = int(min(a.cols - int64_t(cb) * kMxCols, int64_t(kMxCols)));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int p = 0; p < 4; ++p) put(h * 4 + p, staged.row(p * 16 + r0) + col, true);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t r = int64_t(rb) * kMxRows + h * 64 + i * 8 + warp;
        if (r < a.rows)
          staged.store(i * 8 + warp, dst + r * a.row_stride + int64_t(cb) * kMxCols, n);
      }
      __syncthreads();
    }
  } else {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int64_t r = int64_t(rb) * kMxRows + p * 16 + r0;
      put(p, dst + r * a.row_stride + c0, r < a.rows);
    }
  }
}

template <typename T, int ALIGN>
void launch_rows_by(const QuantArgs& a, unsigned grid, cudaStream_t st) {
  if (a.row_index != nullptr)
    quantize_rows_kernel<T, ALIGN, true><<<grid, kThreads, 0, st>>>(a);
  else
    quantize_rows_kernel<T, ALIGN, false><<<grid, kThreads, 0, st>>>(a);
}

template <typename T>
void launch_rows(const QuantArgs& a, int align, unsigned grid, cudaStream_t st) {
  if (align == 16)
    launch_rows_by<T, 16>(a, grid, st);
  else if (align == 8)
    launch_rows_by<T, 8>(a, grid, st);
  else if (align == 4)
    launch_rows_by<T, 4>(a, grid, st);
  else
    launch_rows_by<T, sizeof(T)>(a, grid, st);
}

template <typename T>
fo_status launch_cols(const QuantArgs& a, unsigned grid, cudaStream_t st) {
  constexpr int bytes = TileOf<T>::kBytes;
  if (cudaFuncSetAttribute(quantize_cols_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           bytes) != cudaSuccess)
    return FO_ERR_CUDA;
  quantize_cols_kernel<T><<<grid, kThreads, bytes, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace

fo_status launch_mx_quantize(const void* src, fo_type type, int64_t batch, int64_t batch_stride,
                             int64_t rows, int64_t cols, int64_t row_stride, bool transpose,
                             const int32_t* row_index, int64_t src_rows, void* codes,
                             void* scales, void* stream) {
  const int64_t rb = mx_up(rows, kMxRows) / kMxRows, cb = mx_up(cols, kMxCols) / kMxCols;
  const int64_t blocks = batch * rb * cb;
  if (blocks == 0) return FO_OK;
  if (blocks >= (int64_t(1) << 31)) return FO_ERR_UNSUPPORTED;
  QuantArgs a{src,  batch_stride, row_stride, rows, cols, row_index, src_rows,
              static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), int32_t(rb),
              int32_t(cb)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (transpose)
    return type == FO_TYPE_BF16 ? launch_cols<uint16_t>(a, unsigned(blocks), st)
                                : launch_cols<float>(a, unsigned(blocks), st);
  const unsigned grid = unsigned(blocks);
  const int align = rows_align(src, batch, batch_stride, row_stride, type == FO_TYPE_BF16 ? 2 : 4);
  if (type == FO_TYPE_BF16)
    launch_rows<uint16_t>(a, align, grid, st);
  else
    launch_rows<float>(a, align, grid, st);
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

fo_status launch_mx_dequantize(const void* codes, const void* scales, int64_t batch,
                               int64_t rows, int64_t cols, void* dst, fo_type type,
                               int64_t batch_stride, int64_t row_stride, void* stream) {
  const int64_t rb = mx_up(rows, kMxRows) / kMxRows, cb = mx_up(cols, kMxCols) / kMxCols;
  const int64_t blocks = batch * rb * cb;
  if (blocks == 0) return FO_OK;
  if (blocks >= (int64_t(1) << 31)) return FO_ERR_UNSUPPORTED;
  DequantArgs a{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), dst,
                batch_stride, row_stride, rows, cols, int32_t(rb), int32_t(cb)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = unsigned(blocks);
  const bool staged =
      rows_align(dst, batch, batch_stride, row_stride, type == FO_TYPE_BF16 ? 2 : 4) != 16;
  if (type == FO_TYPE_BF16)
    (staged ? dequantize_kernel<uint16_t, true>
            : dequantize_kernel<uint16_t, false>)<<<grid, kThreads, 0, st>>>(a);
  else
    (staged ? dequantize_kernel<float, true>
            : dequantize_kernel<float, false>)<<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace fo
