// The product of two matrices in the microscaled 4-bit form:
//   D[m][n] = sum_k a[m][k] b[n][k],  a = code value * scale, in fp32,
// for all rows of A or for one range of rows per expert.
//
// The plain first form: a 64 x 64 tile per CTA, blocks of 32 columns decoded
// to fp32 in shared memory, 4 x 4 sums per thread.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "moe_internal.h"
#include "mx_common.cuh"

namespace fo {

namespace {

struct MxGemmArgs {
  const uint8_t *a_codes, *a_scales, *b_codes, *b_scales;
  int64_t M, N, K, k_blocks, n_row_blocks;
  int32_t n_groups;
  const int32_t* first;
  const int32_t* rows;
  void* d;
  int64_t stride;
  int32_t bf16;
  int32_t* status;
};

// One block of 32 columns of a row as fp32 into dst.
__device__ void decode_block(const uint8_t* codes, const uint8_t* scales, int64_t row,
                             int64_t k_blocks, int64_t kb, float* dst, int pitch) {
  const uint8_t s = scales[((row / 128) * k_blocks + kb / 4) * 512 + mx_scale_row(int(row % 128)) +
                           kb % 4];
  const float scale = mx_scale_value(s);
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes + row * (k_blocks * 64) + kb * 16);
  for (int o = 0; o < 4; ++o) {
    uint32_t h[4];
    mx_decode8(c[o], h);
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      dst[(o * 8 + 2 * i) * pitch] = f.x * scale;
      dst[(o * 8 + 2 * i + 1) * pitch] = f.y * scale;
    }
  }
}

__global__ void __launch_bounds__(256) mx_gemm_kernel(const MxGemmArgs a) {
  __shared__ float as[32][65], bs[32][65];
  const int g = blockIdx.z;
  int64_t first = 0, rows = a.M;
  if (a.n_groups > 0) {
    first = a.first[g];
    rows = a.rows[g];
    if (first < 0 || rows < 0 || first % 128 || first + rows > a.M) {
      if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0)
        atomicCAS(a.status, 0, int32_t(FO_ERR_ARG));
      return;
    }
  }
  const int64_t n0 = int64_t(blockIdx.x) * 64;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  for (int64_t m0 = int64_t(blockIdx.y) * 64; m0 < rows; m0 += int64_t(gridDim.y) * 64) {
    float acc[4][4] = {};
    for (int64_t kb = 0; kb < (a.K + 31) / 32; ++kb) {
      __syncthreads();
      if (threadIdx.x < 64) {
        decode_block(a.a_codes, a.a_scales, first + m0 + threadIdx.x, a.k_blocks, kb,
                     &as[0][threadIdx.x], 65);
      } else if (threadIdx.x < 128) {
        const int r = threadIdx.x - 64;
        decode_block(a.b_codes, a.b_scales, g * a.n_row_blocks * 128 + n0 + r, a.k_blocks, kb,
                     &bs[0][r], 65);
      }
      __syncthreads();
      for (int k = 0; k < 32; ++k)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) acc[i][j] += as[k][ty * 4 + i] * bs[k][tx * 4 + j];
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
        if (m >= rows || n >= a.N) continue;
        const int64_t at = (first + m) * a.stride + n;
        if (a.bf16)
          static_cast<__nv_bfloat16*>(a.d)[at] = __float2bfloat16_rn(acc[i][j]);
        else
          static_cast<float*>(a.d)[at] = acc[i][j];
      }
  }
}

}  // namespace

fo_status launch_mx_gemm(int64_t M, int64_t N, int64_t K, const void* a_codes,
                         const void* a_scales, const void* b_codes, const void* b_scales,
                         int32_t n_groups, const int32_t* group_first,
                         const int32_t* group_rows, void* D, fo_type type, int64_t row_stride,
                         int32_t* dev_status, void* stream) {
  if (M == 0 || N == 0) return FO_OK;
  MxGemmArgs a{static_cast<const uint8_t*>(a_codes), static_cast<const uint8_t*>(a_scales),
               static_cast<const uint8_t*>(b_codes), static_cast<const uint8_t*>(b_scales),
               M, N, K, mx_up(K, 128) / 128, mx_up(N, 128) / 128, n_groups, group_first,
               group_rows, D, row_stride, type == FO_TYPE_BF16, dev_status};
  const dim3 grid(unsigned((N + 63) / 64), unsigned(M < 64 * 1024 ? (M + 63) / 64 : 1024),
                  n_groups > 0 ? n_groups : 1);
  mx_gemm_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace fo
