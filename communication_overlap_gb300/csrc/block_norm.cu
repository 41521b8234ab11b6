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

// A row of up to 8192 columns, eight per thread; several rows to a CTA where a row
// has few warps.  CTAs walk over the tokens with the parameters' product in
// registers and DEPTH rows under way in the ring: with a CTA per row, which loads
// its parameters and waits for its own row, 16384 x 4096 took 168 us.
template <typename A, typename S, int DEPTH>
__global__ void __launch_bounds__(1024) norm_kernel(const NormArgs a, int warps) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float buf[2 * 32];
  constexpr int kA = sizeof(A) / 2, kS = sizeof(S) / 2;     // pieces of a row's eight columns
  constexpr int kPieces = kA + kS;
  if (threadIdx.x < 64) buf[threadIdx.x] = 0.0f;
  __syncthreads();
  int turn = 0;
  const RowGroup g = RowGroup::of(warps);
  const OwnRing ring(smem);
  const int col = g.tid * 8;
  const bool has = col < a.hidden;
  const int rows = int(blockDim.x) / (warps * 32);
  const int64_t step = int64_t(gridDim.x) * rows;
  const int64_t t0 = int64_t(blockIdx.x) * rows + g.index;
  const float inv = 1.0f / float(a.hidden);
  const auto fetch = [&](int64_t t, int stage) {
    if (has && t < a.tokens) {
      ring.fetch(stage * kPieces, static_cast<const A*>(a.x) + t * a.x_stride + col);
      if (a.residual != nullptr)
        ring.fetch(stage * kPieces + kA,
                   static_cast<const S*>(a.residual) + t * a.residual_stride + col);
    }
    OwnRing::commit();
  };
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) fetch(t0 + i * step, i);
  float w[8], pre[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pre[i] = 0.0f;
  if (has && a.pre != nullptr) load_param<8>(a.pre, col, a.params_f32, pre);
  int64_t gate_row = -1;
  int stage = 0;
  for (int64_t t = t0; t < a.tokens; t += step) {
    if (has) {
      const int64_t row = a.gate_stride ? int64_t(uint32_t(t) / uint32_t(a.gate_rows)) : 0;
      if (row != gate_row) load_factor(a, col, row * a.gate_stride, w);
      gate_row = row;
    }
    OwnRing::wait<DEPTH - 1>();
    float x[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = s[i] = 0.0f;
    if (has) {
      ring.get<A>(stage * kPieces, x);
      if (a.residual != nullptr) ring.get<S>(stage * kPieces + kA, s);
    }
    fetch(t + DEPTH * step, stage);
    if (++stage == DEPTH) stage = 0;
    float r1 = 1.0f;
    if (a.post != nullptr) {
      float sum[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] = fmaf(x[i], x[i], sum[0]);
      g.sums<1>(sum, buf, turn);
      r1 = rsqrtf(fmaf(sum[0], inv, a.eps));
      if (g.tid == 0) a.post_rstd[t] = r1;
    }
    float sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = fmaf(w[i], x[i] * r1, s[i]);
      sum[0] = fmaf(s[i], s[i], sum[0]);
    }
    if (has && a.sum != nullptr)
      store_piece<8>(static_cast<S*>(a.sum) + t * a.sum_stride + col, s);
    if (a.pre == nullptr) continue;
    g.sums<1>(sum, buf, turn);
    const float r2 = rsqrtf(fmaf(sum[0], inv, a.eps));
    if (g.tid == 0) a.pre_rstd[t] = r2;
    if (!has) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] *= r2 * pre[i];
    store_piece<8>(static_cast<A*>(a.y) + t * a.y_stride + col, s);
  }
  OwnRing::wait<0>();
}

// Any row: a CTA per token, W columns per thread at a time.
template <typename A, typename S, int W>
__global__ void __launch_bounds__(512) norm_any_kernel(const NormArgs a) {
  __shared__ float buf[2 * 32];
  int turn = 0;
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
    cta_sums<1>(sum, buf, turn);
    r1 = rsqrtf(fmaf(sum[0], 1.0f / float(a.hidden), a.eps));
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
    cta_sums<1>(sum, buf, turn);
    r2 = rsqrtf(fmaf(sum[0], 1.0f / float(a.hidden), a.eps));
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

template <typename A, typename S, int DEPTH>
fo_status launch_ring(const NormArgs& a, int warps, int rows, int row_bytes, cudaStream_t st) {
  int sms = 0;
  fo_status q = sm_count(&sms);
  if (q == FO_OK) q = allow_smem<norm_kernel<A, S, DEPTH>>();
  if (q != FO_OK) return q;
  const int threads = rows * warps * 32;
  const int64_t most = (int64_t(a.tokens) + rows - 1) / rows;
  const int64_t ctas = int64_t(sms) * (threads <= 512 ? 2 : 1);
  norm_kernel<A, S, DEPTH><<<unsigned(most < ctas ? most : ctas), threads, DEPTH * row_bytes, st>>>(
      a, warps);
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

template <typename A, typename S>
fo_status launch(const NormArgs& a, bool vec, cudaStream_t st) {
  if (vec && a.hidden <= 8192) {
    const int warps = (a.hidden + 255) / 256, rows = rows_of_cta(warps, 16);
    const int threads = rows * warps * 32;
    // four rows under way where two CTAs of up to 512 threads fit on an SM so, else two
    const int row = threads * 16 * int(sizeof(A) + sizeof(S)) / 2;
    const bool deep = 4 * row <= (threads <= 512 ? kNormSmem / 2 : kNormSmem);
    return deep ? launch_ring<A, S, 4>(a, warps, rows, row, st)
                : launch_ring<A, S, 2>(a, warps, rows, row, st);
  } else if (vec) {
    norm_any_kernel<A, S, 8><<<unsigned(a.tokens), 512, 0, st>>>(a);
  } else {
    const int warps = (a.hidden + 31) / 32;
    norm_any_kernel<A, S, 1><<<unsigned(a.tokens), (warps < 16 ? warps : 16) * 32, 0, st>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace

fo_status launch_block_norm(const NormArgs& a, fo_type type, fo_type stream_type, void* stream) {
  const bool vec = norm_rows_on_16(a, type, stream_type);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (type == FO_TYPE_F32) return launch<float, float>(a, vec, st);
  if (stream_type == FO_TYPE_F32) return launch<uint16_t, float>(a, vec, st);
  return launch<uint16_t, uint16_t>(a, vec, st);
}

}  // namespace fo
