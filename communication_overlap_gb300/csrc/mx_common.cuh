// The microscaled 4-bit form (include/fo.h): E2M1 codes, one E8M0 scale per
// 32 values, scales in blocks of 128 rows x 4.
#pragma once

#include <cstdint>

#include "device_common.cuh"

namespace fo {

constexpr int kMxBlock = 32;        // values that share a scale
constexpr int kMxRows = 128;        // rows of a block of scales
constexpr int kMxCols = 128;        // columns of a block of scales
constexpr int kMxScaleBytes = 512;  // bytes of a block of scales

__host__ __device__ __forceinline__ int64_t mx_up(int64_t n, int64_t m) {
  return (n + m - 1) / m * m;
}

// Offset of a row's four scales inside its block of 512 bytes.
__host__ __device__ __forceinline__ int mx_scale_row(int r) {
  return (r & 31) * 16 + (r >> 5) * 4;
}

// The scale's exponent byte from the largest magnitude's bits: floor(log2 a)
// is the exponent field (0 for zeros and subnormals, far below the smallest
// scale), so the byte is that field - 2, at least 0; 255 for infinity or NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  if (e == 255u) return 255u;
  return e > 2u ? e - 2u : 0u;
}

// 2^(127 - s): the factor that divides a value by its scale, exact.
__device__ __forceinline__ float mx_inverse_scale(uint32_t s) {
  return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
}

// 2^(s - 127), NaN for 255.
__device__ __forceinline__ float mx_scale_value(uint32_t s) {
  if (s == 255u) return __uint_as_float(0x7fffffffu);
  return s == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23);
}

// Eight values already divided by their scale -> eight codes, value 0 in the
// low nibble: round to nearest, ties to even, magnitudes above 6 to 6.
__device__ __forceinline__ uint32_t mx_encode8(const float (&v)[8]) {
  uint32_t out;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(out)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return out;
}

// Eight codes -> their E2M1 values as four f16 pairs (exact).
__device__ __forceinline__ void mx_decode8(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

}  // namespace fo
