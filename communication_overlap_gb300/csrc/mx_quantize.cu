// Conversion to and from the microscaled 4-bit form.
//
// Per block of 32 values x_i of a row, with a = max |x_i|:
//   s = 2^(floor(log2 a) - 2),  q_i = the E2M1 value nearest x_i / s.
// floor(log2 a) is a's exponent field and s a power of two, so s and x_i / s
// are exact and the only rounding is the one to E2M1.
//
// Both directions move each byte once and compute almost nothing: HBM bounds
// them.  A CTA takes one block of scales (128 rows x 128 columns): 256
// threads, each 8 rows apart x 8 columns, all loads issued before the first
// use (16 bytes x 8 per thread of bf16), four neighbouring lanes to a block of
// 32.
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
  __device__ __forceinline__ void load(const T* p) {   // 16-byte aligned
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
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

// Rows of the source (or gathered rows of it) become rows of the result.
template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantArgs a) {
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
  constexpr uintptr_t kAlign = 15;
  const bool vec = ((reinterpret_cast<uintptr_t>(src) |
                     uintptr_t(a.row_stride) * sizeof(T)) & kAlign) == 0;
  const int r0 = threadIdx.x >> 4;                 // 16 rows per pass
  uint8_t* codes = a.codes + (b * a.row_blocks + rb) * int64_t(kMxRows) * (int64_t(a.col_blocks) * 64);
  // which rows, then all loads, then the rest: no load waits for another
  const T* from[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int64_t r = int64_t(rb) * kMxRows + p * 16 + r0;
    int64_t row = r < a.rows ? r : -1;
    if (a.row_index != nullptr && r < a.rows) {
      row = a.row_index[r];
      if (row >= a.src_rows) row = -1;
    }
    from[p] = row < 0 ? nullptr : src + row * a.row_stride + c0;
  }
  Eight<T> v[8];
  if (vec && valid == 8) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      v[p].zero();
      if (from[p] != nullptr) v[p].load(from[p]);
    }
  } else {
#pragma unroll
    for (int p = 0; p < 8; ++p) v[p].load_some(from[p], from[p] != nullptr ? valid : 0);
  }
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
    for (int i = 0; i < 8; ++i) u[i] = s == 255u ? 0.0f : v[p].value(i) * inv;
    __stcs(reinterpret_cast<uint32_t*>(codes + int64_t(r) * (int64_t(a.col_blocks) * 64) +
                                       int64_t(cb) * 64 + col / 2),
           mx_encode8(u));
    if ((threadIdx.x & 3) == 0)
      reinterpret_cast<uint8_t*>(scale_block)[mx_scale_row(r) + (col >> 5)] = uint8_t(s);
  }
  __syncthreads();
  if (threadIdx.x < kMxScaleBytes / 4)
    reinterpret_cast<uint32_t*>(a.scales +
                                ((b * a.row_blocks + rb) * a.col_blocks + cb) *
                                    int64_t(kMxScaleBytes))[threadIdx.x] = scale_block[threadIdx.x];
}

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
  uint32_t m0 = 0, m1 = 0;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) {
    uint32_t x0, x1;
    if constexpr (sizeof(T) == 2) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(from + i * C::kPitch);
      x0 = w << 16, x1 = w & 0xffff0000u;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(from + i * C::kPitch);
      x0 = w.x, x1 = w.y;
    }
    m0 = max(m0, x0 & 0x7fffffffu);
    m1 = max(m1, x1 & 0x7fffffffu);
  }
  const uint32_t s0 = mx_scale_byte(m0), s1 = mx_scale_byte(m1);
  const float i0 = mx_inverse_scale(s0), i1 = mx_inverse_scale(s1);
  uint32_t q0[4], q1[4];
#pragma unroll
  for (int o = 0; o < 4; ++o) {
    float u0[8], u1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x0, x1;
      if constexpr (sizeof(T) == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(from + (o * 8 + i) * C::kPitch);
        x0 = bf16lo(w), x1 = bf16hi(w);
      } else {
        const float2 w = *reinterpret_cast<const float2*>(from + (o * 8 + i) * C::kPitch);
        x0 = w.x, x1 = w.y;
      }
      u0[i] = s0 == 255u ? 0.0f : x0 * i0;
      u1[i] = s1 == 255u ? 0.0f : x1 * i1;
    }
    q0[o] = mx_encode8(u0);
    q1[o] = mx_encode8(u1);
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

template <typename T>
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
  const bool vec = valid == 8 && ((reinterpret_cast<uintptr_t>(dst) |
                                   uintptr_t(a.row_stride) * sizeof(T)) & 15) == 0;
  const int r0 = threadIdx.x >> 4;
  const int64_t pitch = int64_t(a.col_blocks) * 64;
  const uint8_t* codes = a.codes + (b * a.row_blocks + rb) * int64_t(kMxRows) * pitch +
                         int64_t(cb) * 64 + col / 2;
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
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int64_t r = int64_t(rb) * kMxRows + p * 16 + r0;
    if (r >= a.rows) continue;
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
    T* to = dst + r * a.row_stride + c0;
    if constexpr (sizeof(T) == 2) {
      const uint4 w = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      if (vec) {
        __stcs(reinterpret_cast<uint4*>(to), w);
      } else {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < valid) to[i] = uint16_t(u[i / 2] >> (16 * (i & 1)));
      }
    } else {
      if (vec) {
        __stcs(reinterpret_cast<float4*>(to), make_float4(v[0], v[1], v[2], v[3]));
        __stcs(reinterpret_cast<float4*>(to) + 1, make_float4(v[4], v[5], v[6], v[7]));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < valid) to[i] = v[i];
      }
    }
  }
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
  if (type == FO_TYPE_BF16)
    quantize_rows_kernel<uint16_t><<<unsigned(blocks), kThreads, 0, st>>>(a);
  else
    quantize_rows_kernel<float><<<unsigned(blocks), kThreads, 0, st>>>(a);
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
  if (type == FO_TYPE_BF16)
    dequantize_kernel<uint16_t><<<unsigned(blocks), kThreads, 0, st>>>(a);
  else
    dequantize_kernel<float><<<unsigned(blocks), kThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace fo
