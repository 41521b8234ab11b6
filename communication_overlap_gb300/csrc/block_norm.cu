// RMS norm after a block, its gate and scale into the residual stream, and RMS
// norm before the next block, in one pass:
//
//   u = x r1 post,   r1 = 1 / sqrt(mean x^2 + eps)    (u = x without post)
//   s = residual + scale gate u                       (the stream)
//   y = s r2 pre,    r2 = 1 / sqrt(mean s^2 + eps)
//
// A row of up to 8192 columns on 16 bytes stays in registers between its loads
// and its stores, so each tensor moves once and HBM bounds the kernel; s enters
// y before it is rounded.  Other rows are walked column by column, once per sum
// and once for y.
#include <cuda_runtime.h>

#include "block_norm.cuh"

namespace fo {

namespace {

// u of W columns, then s.
template <int W>
__device__ __forceinline__ void stream_of(const NormArgs& a, int col, int64_t gate_row, float r1,
                                          const float (&x)[W], const float (&r)[W],
                                          float (&s)[W]) {
  float v[W], p[W];
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = x[i];
  if (a.post != nullptr) {
    load_param<W>(a.post, col, a.params_f32, p);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = v[i] * r1 * p[i];
  }
  if (a.gate != nullptr) {
    load_param<W>(a.gate, gate_row + col, a.params_f32, p);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] *= p[i];
  }
#pragma unroll
  for (int i = 0; i < W; ++i) s[i] = fmaf(a.scale, v[i], r[i]);
}

// One round of eight columns per thread; several rows to a CTA where a row has up
// to four warps.
template <typename A, typename S>
__global__ void __launch_bounds__(1024) norm_kernel(const NormArgs a, int warps, int rows) {
  __shared__ float buf[2 * 32];
  int turn = 0;
  const int row = int(threadIdx.x >> 5) / warps;
  const int tid = int(threadIdx.x) - row * warps * 32, col = tid * 8;
  const int64_t t = int64_t(blockIdx.x) * rows + row;
  const bool live = t < a.tokens && col < a.hidden;
  Piece<A, 8> px;
  Piece<S, 8> pr;
  px.load(static_cast<const A*>(a.x) + t * a.x_stride + col, live);
  pr.load(static_cast<const S*>(a.residual) + t * a.residual_stride + col,
          live && a.residual != nullptr);
  float x[8], r[8], s[8];
  px.get(x);
  float r1 = 1.0f;
  if (a.post != nullptr) {
    float sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[0] = fmaf(x[i], x[i], sum[0]);
    row_sums<1>(sum, row * warps, warps, buf, turn);
    r1 = 1.0f / sqrtf(sum[0] / float(a.hidden) + a.eps);
    if (live && tid == 0) a.post_rstd[t] = r1;
  }
  pr.get(r);
  float sum[1] = {0.0f};
  if (live) {
    stream_of<8>(a, col, a.gate ? t / a.gate_rows * a.gate_stride : 0, r1, x, r, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[0] = fmaf(s[i], s[i], sum[0]);
    if (a.sum != nullptr) store_piece<8>(static_cast<S*>(a.sum) + t * a.sum_stride + col, s);
  }
  if (a.pre == nullptr) return;
  row_sums<1>(sum, row * warps, warps, buf, turn);
  if (!live) return;
  const float r2 = 1.0f / sqrtf(sum[0] / float(a.hidden) + a.eps);
  if (tid == 0) a.pre_rstd[t] = r2;
  float p[8], y[8];
  load_param<8>(a.pre, col, a.params_f32, p);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = s[i] * r2 * p[i];
  store_piece<8>(static_cast<A*>(a.y) + t * a.y_stride + col, y);
}

// Any row: a CTA per token, W columns per thread at a time.
template <typename A, typename S, int W>
__global__ void __launch_bounds__(512) norm_any_kernel(const NormArgs a) {
  __shared__ float buf[2 * 32];
  int turn = 0;
  const int warps = int(blockDim.x) >> 5;
  const int64_t t = blockIdx.x;
  const A* x = static_cast<const A*>(a.x) + t * a.x_stride;
  const S* residual = static_cast<const S*>(a.residual) + t * a.residual_stride;
  const int64_t gate_row = a.gate ? t / a.gate_rows * a.gate_stride : 0;
  const int step = int(blockDim.x) * W;
  float r1 = 1.0f;
  if (a.post != nullptr) {
    float sum[1] = {0.0f};
    for (int col = int(threadIdx.x) * W; col < a.hidden; col += step) {
      Piece<A, W> p;
      float v[W];
      p.load(x + col, true);
      p.get(v);
#pragma unroll
      for (int i = 0; i < W; ++i) sum[0] = fmaf(v[i], v[i], sum[0]);
    }
    row_sums<1>(sum, 0, warps, buf, turn);
    r1 = 1.0f / sqrtf(sum[0] / float(a.hidden) + a.eps);
    if (threadIdx.x == 0) a.post_rstd[t] = r1;
  }
  const auto stream = [&](int col, float (&s)[W]) {
    Piece<A, W> px;
    Piece<S, W> pr;
    float v[W], r[W];
    px.load(x + col, true);
    pr.load(residual + col, a.residual != nullptr);
    px.get(v);
    pr.get(r);
    stream_of<W>(a, col, gate_row, r1, v, r, s);
  };
  float sum[1] = {0.0f};
  float r2 = 1.0f;
  if (a.pre != nullptr) {
    for (int col = int(threadIdx.x) * W; col < a.hidden; col += step) {
      float s[W];
      stream(col, s);
#pragma unroll
      for (int i = 0; i < W; ++i) sum[0] = fmaf(s[i], s[i], sum[0]);
    }
    row_sums<1>(sum, 0, warps, buf, turn);
    r2 = 1.0f / sqrtf(sum[0] / float(a.hidden) + a.eps);
    if (threadIdx.x == 0) a.pre_rstd[t] = r2;
  }
  for (int col = int(threadIdx.x) * W; col < a.hidden; col += step) {
    float s[W];
    stream(col, s);
    if (a.sum != nullptr) store_piece<W>(static_cast<S*>(a.sum) + t * a.sum_stride + col, s);
    if (a.pre != nullptr) {
      float p[W];
      load_param<W>(a.pre, col, a.params_f32, p);
#pragma unroll
      for (int i = 0; i < W; ++i) s[i] = s[i] * r2 * p[i];
      store_piece<W>(static_cast<A*>(a.y) + t * a.y_stride + col, s);
    }
  }
}

template <typename A, typename S>
void launch(const NormArgs& a, bool vec, cudaStream_t st) {
  if (vec && a.hidden <= 8192) {
    const int warps = (a.hidden + 255) / 256, rows = warps <= 4 ? 8 / warps : 1;
    const unsigned grid = unsigned((int64_t(a.tokens) + rows - 1) / rows);
    norm_kernel<A, S><<<grid, rows * warps * 32, 0, st>>>(a, warps, rows);
  } else if (vec) {
    norm_any_kernel<A, S, 8><<<unsigned(a.tokens), 512, 0, st>>>(a);
  } else {
    const int warps = (a.hidden + 31) / 32;
    norm_any_kernel<A, S, 1><<<unsigned(a.tokens), (warps < 16 ? warps : 16) * 32, 0, st>>>(a);
  }
}

}  // namespace

fo_status launch_block_norm(const NormArgs& a, fo_type type, fo_type stream_type, void* stream) {
  const bool vec = norm_rows_on_16(a, type, stream_type);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (type == FO_TYPE_F32)
    launch<float, float>(a, vec, st);
  else if (stream_type == FO_TYPE_F32)
    launch<uint16_t, float>(a, vec, st);
  else
    launch<uint16_t, uint16_t>(a, vec, st);
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace fo
