// RMS norm after a block, its gate and scale into the residual stream, and RMS
// norm before the next block, in one pass:
//
//   u = x r1 post,   r1 = 1 / sqrt(mean x^2 + eps)    (u = x without post)
//   s = residual + scale gate u                       (the stream)
//   y = s r2 pre,    r2 = 1 / sqrt(mean s^2 + eps)
//
// A row of up to 8192 columns on 16 bytes stays in registers between its loads
// and its stores, so each tensor moves once and HBM bounds the kernel; s enters
// y before it is rounded; so do rows of up to 4096 columns that lie anyhow.  Longer
// ones are walked along, once per sum and once for y.
//
// 16384 x 4096 of bf16: 537 MB in 84 us (6.4 TB/s).  Few or short rows leave each CTA a
// few rows only, and launch, the first row's way and the last CTA's weigh more: 4095 x
// 2752 of bf16 into an fp32 stream 135 MB in 30 us (4.5).  One row of 4096 takes 3.3 us.
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

// A worker's tokens: with several rows of the gate next to each other, so that it meets
// few of them (their factors are a wait each: five sequences of 819 x 2752 33 -> 30 us),
// else at a stride (16384 x 4096 in bf16 92 us, next to each other 98).
struct Tokens {
  int first, end, step;
  __device__ __forceinline__ Tokens(const NormArgs& a, int worker, int workers) {
    if (a.gate_stride == 0) {
      first = worker, end = a.tokens, step = workers;
    } else {
      const int each = a.tokens / workers, more = a.tokens % workers;
      first = worker * each + min(worker, more);
      end = first + each + (worker < more ? 1 : 0);
      step = 1;
    }
  }
};

// Rows of up to 8192 columns; several to a CTA where they have few warps.  CTAs walk
// over the tokens with the parameters' product in registers and DEPTH rows under way
// in the ring, two values per instruction.  16384 x 4096: a CTA per row, which loads
// its parameters and waits for its own row, took 168 us; this with eight columns per
// thread and one value per instruction 116.
template <typename A, typename S, int NV, int DEPTH>
__global__ void __launch_bounds__(512, 1) norm_kernel(const NormArgs a, int warps) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float buf[2 * 32];
  constexpr int kA = sizeof(A) / 2, kS = sizeof(S) / 2;     // pieces of eight columns
  constexpr int kPieces = NV * (kA + kS);
  if (threadIdx.x < 64) buf[threadIdx.x] = 0.0f;
  __syncthreads();
  int turn = 0;
  const RowGroup g = RowGroup::of(warps);
  const OwnRing ring(smem);
  const int rows = int(blockDim.x) / (warps * 32);
  const Tokens own(a, int(blockIdx.x) * rows + g.index, int(gridDim.x) * rows);
  const int t0 = own.first;
  const float inv = 1.0f / float(a.hidden);
  int col[NV];
  bool has[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    col[v] = (v * warps * 32 + g.tid) * 8;
    has[v] = col[v] < a.hidden;
  }
  const A* x_at = static_cast<const A*>(a.x) + int64_t(t0) * a.x_stride;
  const S* r_at = static_cast<const S*>(a.residual) + int64_t(t0) * a.residual_stride;
  const int64_t x_step = own.step * a.x_stride, r_step = own.step * a.residual_stride;
  int fetched = t0;
  const auto fetch = [&](int stage) {
    if (fetched < own.end) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int at = stage * kPieces + v * (kA + kS);
        ring.fetch(at, x_at, col[v], a.hidden);
        if (a.residual != nullptr) ring.fetch(at + kA, r_at, col[v], a.hidden);
        if (has[v]) prefetch_gate(a, fetched, col[v]);
      }
    }
    OwnRing::commit();
    fetched += own.step;
    x_at += x_step;
    r_at += r_step;
  };
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) fetch(i);
  Pair w[NV][4], pre[NV][4];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = 0.0f;
    if (has[v] && a.pre != nullptr) load_param<8>(a.pre, col[v], a.params_f32, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) pre[v][i] = Pair::of(p[2 * i], p[2 * i + 1]), w[v][i] = Pair::of(0.0f);
  }
  int gate_row = -1, stage = 0;
  S* sum_at = static_cast<S*>(a.sum) + int64_t(t0) * a.sum_stride;
  A* y_at = static_cast<A*>(a.y) + int64_t(t0) * a.y_stride;
  const int64_t sum_step = own.step * a.sum_stride, y_step = own.step * a.y_stride;
  for (int t = t0; t < own.end; t += own.step) {
    const int row = a.gate_stride ? int(uint32_t(t) / uint32_t(a.gate_rows)) : 0;
    if (row != gate_row) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float p[8];
        if (!has[v]) continue;
        load_factor(a, col[v], row * a.gate_stride, p);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[v][i] = Pair::of(p[2 * i], p[2 * i + 1]);
      }
      gate_row = row;
    }
    OwnRing::wait<DEPTH - 1>();
    Pair x[NV][4], s[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[v][i] = s[v][i] = Pair::of(0.0f);
      if (has[v]) {
        const int at = stage * kPieces + v * (kA + kS);
        get_pairs<A>(ring, at, x[v]);
        if (a.residual != nullptr) get_pairs<S>(ring, at + kA, s[v]);
      }
    }
    fetch(stage);
    stage = stage + 1 == DEPTH ? 0 : stage + 1;
    Pair r1 = Pair::of(1.0f);
    if (a.post != nullptr) {
      Pair sum = Pair::of(0.0f);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = fma2(x[v][i], x[v][i], sum);
      }
      float total[1] = {sum.sum()};
      g.sums<1>(total, buf, turn);
      const float r = rsqrtf(fmaf(total[0], inv, a.eps));
      if (g.tid == 0) a.post_rstd[t] = r;
      r1 = Pair::of(r);
    }
    Pair sum = Pair::of(0.0f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[v][i] = fma2(w[v][i], x[v][i] * r1, s[v][i]);
        sum = fma2(s[v][i], s[v][i], sum);
      }
      if (a.sum != nullptr) store8_warp(sum_at + col[v], has[v], s[v]);
    }
    sum_at += sum_step;
    if (a.pre == nullptr) continue;
    float total[1] = {sum.sum()};
    g.sums<1>(total, buf, turn);
    const float r2 = rsqrtf(fmaf(total[0], inv, a.eps));
    if (g.tid == 0) a.pre_rstd[t] = r2;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[v][i] = s[v][i] * Pair::of(r2) * pre[v][i];
      store8_warp(y_at + col[v], has[v], s[v]);
    }
    y_at += y_step;
  }
  OwnRing::wait<0>();
}

// Rows of up to 4096 columns that need not lie on 16 bytes: eight columns per thread,
// E neighbouring ones of each 32 E of the row's threads, so that a warp's loads are of
// neighbouring addresses; the next row is loaded while one is worked on.  (Walked
// column by column, three times: 342 us for 16384 x 4095 of bf16.)
template <typename A, typename S, int E>
__global__ void __launch_bounds__(512, 1) norm_few_kernel(const NormArgs a, int warps) {
  constexpr int U = 8 / E;
  __shared__ __align__(16) float buf[2 * 32];
  if (threadIdx.x < 64) buf[threadIdx.x] = 0.0f;
  __syncthreads();
  int turn = 0;
  const RowGroup g = RowGroup::of(warps);
  const int rows = int(blockDim.x) / (warps * 32);
  const Tokens own(a, int(blockIdx.x) * rows + g.index, int(gridDim.x) * rows);
  const int first = g.tid * E, stride = warps * 32 * E;
  const float inv = 1.0f / float(a.hidden);
  Few<A, E> px[U];
  Few<S, E> pr[U];
  const auto load = [&](int64_t t) {
    const A* x = static_cast<const A*>(a.x) + t * a.x_stride + first;
    const S* r = static_cast<const S*>(a.residual) + t * a.residual_stride + first;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool has = t < own.end && first + i * stride < a.hidden;
      px[i].zero();
      pr[i].zero();
      if (has) px[i].load(x + i * stride);
      if (has && a.residual != nullptr) pr[i].load(r + i * stride);
    }
  };
  load(own.first);
  float w[U][E], pre[U][E];
#pragma unroll
  for (int i = 0; i < U; ++i) {
#pragma unroll
    for (int e = 0; e < E; ++e) w[i][e] = pre[i][e] = 0.0f;
    if (a.pre != nullptr && first + i * stride < a.hidden)
      load_few_param<E>(a.pre, first + i * stride, a.params_f32, pre[i]);
  }
  int gate_row = -1;
  for (int t = own.first; t < own.end; t += own.step) {
    const int row = a.gate_stride ? int(uint32_t(t) / uint32_t(a.gate_rows)) : 0;
    if (row != gate_row) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (first + i * stride < a.hidden)
          load_few_factor<E>(a, first + i * stride, row * a.gate_stride, w[i]);
      gate_row = row;
    }
    float x[U][E], s[U][E], r1 = 1.0f, sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < U; ++i) {
      px[i].get(x[i]);
      pr[i].get(s[i]);
    }
    load(int64_t(t) + own.step);
    if (a.post != nullptr) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
#pragma unroll
        for (int e = 0; e < E; ++e) sum[0] = fmaf(x[i][e], x[i][e], sum[0]);
      }
      g.sums<1>(sum, buf, turn);
      r1 = rsqrtf(fmaf(sum[0], inv, a.eps));
      if (g.tid == 0) a.post_rstd[t] = r1;
      sum[0] = 0.0f;
    }
    S* to = static_cast<S*>(a.sum) + t * a.sum_stride + first;
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        s[i][e] = fmaf(w[i][e], x[i][e] * r1, s[i][e]);
        sum[0] = fmaf(s[i][e], s[i][e], sum[0]);
      }
      if (a.sum != nullptr && first + i * stride < a.hidden)
        Few<S, E>::store(to + i * stride, s[i]);
    }
    if (a.pre == nullptr) continue;
    g.sums<1>(sum, buf, turn);
    const float r2 = rsqrtf(fmaf(sum[0], inv, a.eps));
    if (g.tid == 0) a.pre_rstd[t] = r2;
    A* y = static_cast<A*>(a.y) + t * a.y_stride + first;
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int e = 0; e < E; ++e) s[i][e] = s[i][e] * r2 * pre[i][e];
      if (first + i * stride < a.hidden) Few<A, E>::store(y + i * stride, s[i]);
    }
  }
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

template <typename A, typename S, int NV, int DEPTH>
fo_status launch_ring(const NormArgs& a, const RowShape& s, int row_bytes, cudaStream_t st) {
  int sms = 0;
  fo_status q = sm_count(&sms);
  if (q == FO_OK) q = allow_smem<norm_kernel<A, S, NV, DEPTH>>();
  if (q != FO_OK) return q;
  const int64_t most = (int64_t(a.tokens) + s.rows - 1) / s.rows;
  const int64_t ctas = int64_t(sms) * (s.threads <= 256 ? 2 : 1);
  norm_kernel<A, S, NV, DEPTH>
      <<<unsigned(most < ctas ? most : ctas), s.threads, DEPTH * row_bytes, st>>>(a, s.warps);
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

template <typename A, typename S>
fo_status launch(const NormArgs& a, bool vec, bool two, cudaStream_t st) {
  if (vec && a.hidden <= 8192) {
    // two times eight columns per thread where a row has more than 256 (half the threads
    // to meet at its sums, half the addresses), and CTAs of 256 threads where that does
    const RowShape s = row_shape(a.hidden, a.hidden <= 256 ? 1 : 2, 8);
    // four rows under way where two CTAs of 256 threads, or one of more, fit so, else two
    const int row = s.threads * s.nv * 16 * int(sizeof(A) + sizeof(S)) / 2;
    const bool deep = 4 * row <= (s.threads <= 256 ? kBlockSmem / 2 : kBlockSmem);
    if (s.nv == 1) return launch_ring<A, S, 1, 4>(a, s, row, st);
    if constexpr (sizeof(A) == 4) {       // (of bf16 rows four always fit)
      if (!deep) return launch_ring<A, S, 2, 2>(a, s, row, st);
    }
    return launch_ring<A, S, 2, 4>(a, s, row, st);
  } else if (!vec && a.hidden <= 4096) {
    int sms = 0;
    const fo_status q = sm_count(&sms);
    if (q != FO_OK) return q;
    const RowShape s = row_shape(a.hidden, 1, 16);
    const int64_t most = (int64_t(a.tokens) + s.rows - 1) / s.rows;
    const unsigned grid = unsigned(most < sms ? most : sms);
    if (two)
      norm_few_kernel<A, S, 2><<<grid, s.threads, 0, st>>>(a, s.warps);
    else
      norm_few_kernel<A, S, 1><<<grid, s.threads, 0, st>>>(a, s.warps);
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
  const bool two = norm_rows_on_two(a, type, stream_type);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (type == FO_TYPE_F32) return launch<float, float>(a, vec, two, st);
  if (stream_type == FO_TYPE_F32) return launch<uint16_t, float>(a, vec, two, st);
  return launch<uint16_t, uint16_t>(a, vec, two, st);
}

}  // namespace fo
