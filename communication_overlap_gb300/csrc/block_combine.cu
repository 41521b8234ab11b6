// The weighted sum of a token's rows of the experts' outputs, and its gradients.
//
//   y_t = sum over slots s of w_ts rows[r_ts],  r = token_row (-1: no row)
//   drows[r_ts] = w_ts dy_t,  dw_ts = <dy_t, rows[r_ts]>,  drows = 0 elsewhere.
//
// Both move each byte once and HBM bounds them.  Sums are fp32, in slot order;
// outputs are rounded once.
#include <cuda_runtime.h>

#include "block_common.cuh"

namespace fo {

namespace {

constexpr int kThreads = 256;

struct CombineArgs {
  const void* rows;
  int64_t row_stride, table_rows;
  const int32_t* token_row;
  const float* weights;    // NULL: ones
  int64_t tokens;
  int32_t hidden, top_k;
  void* y;
  int64_t y_stride;
  int32_t* status;
  // the shape of the grid
  int32_t pieces;          // CTAs along a token's columns
  int32_t per_cta;         // tokens of a CTA
  int32_t chunks;          // threads along a token's columns
};

// The row of a pair, -1 for none; a row outside the table is recorded.
__device__ __forceinline__ int row_of(int32_t r, int64_t table_rows, int32_t* status) {
  if (r < table_rows) return r;
  atomicCAS(status, 0, int32_t(FO_ERR_ARG));
  return -1;
}

// A thread takes eight columns of a token (VEC: rows and y on 16 bytes) or one.
template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs a) {
  constexpr int W = VEC ? 8 : 1;
  const int piece = blockIdx.x % unsigned(a.pieces);
  const int64_t t0 = int64_t(blockIdx.x / unsigned(a.pieces)) * a.per_cta;
  const int local = int(threadIdx.x) / a.chunks;
  const int64_t c = int64_t(piece) * kThreads + (a.pieces > 1 ? int(threadIdx.x)
                                                               : int(threadIdx.x) % a.chunks);
  const int64_t t = t0 + (a.pieces > 1 ? 0 : local);
  if ((a.pieces == 1 && local >= a.per_cta) || t >= a.tokens || c * W >= a.hidden) return;
  const T* rows = static_cast<const T*>(a.rows) + c * W;
  const int32_t* index = a.token_row + t * a.top_k;
  const float* weights = a.weights ? a.weights + t * a.top_k : nullptr;
  float acc[W];
#pragma unroll
  for (int i = 0; i < W; ++i) acc[i] = 0.0f;
  constexpr int kAhead = 4;      // rows under way
  for (int s0 = 0; s0 < a.top_k; s0 += kAhead) {
    int32_t r[kAhead];
    float w[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int s = s0 + j;
      r[j] = s < a.top_k ? row_of(__ldg(index + s), a.table_rows, a.status) : -1;
      w[j] = s < a.top_k && weights ? __ldg(weights + s) : 1.0f;
    }
    if constexpr (VEC) {
      Pack8<T> v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (r[j] >= 0) v[j].load_once(rows + r[j] * a.row_stride);
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (r[j] >= 0) {
          float f[8];
          v[j].get(f);
#pragma unroll
          for (int i = 0; i < W; ++i) acc[i] = fmaf(w[j], f[i], acc[i]);
        }
    } else {
      T v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (r[j] >= 0) v[j] = __ldcs(rows + r[j] * a.row_stride);
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (r[j] >= 0) acc[0] = fmaf(w[j], widen(v[j]), acc[0]);
    }
  }
  O* y = static_cast<O*>(a.y) + t * a.y_stride + c * W;
  if constexpr (VEC)
    store8(y, acc);
  else
    *y = narrow<O>(acc[0]);
}

struct CombineBackArgs {
  CombineArgs f;
  const void* dy;
  int64_t dy_stride;
  const int32_t* row_token;
  void* drows;
  int64_t drows_stride;
  float* dweights;
  int32_t warps;            // of a token: 1, 2, 4 or 8
  int64_t token_ctas;       // the CTAs after these zero the rows without a token
};

// A token per group of warps, its slots four at a time: dy, a row each, the
// products and the row's gradient; then the sums over the group.
template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const CombineBackArgs a) {
  constexpr int W = VEC ? 8 : 1;
  constexpr int kSlots = 4;
  const CombineArgs& f = a.f;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T* drows = static_cast<T*>(a.drows);
  if (blockIdx.x >= a.token_ctas) {
    const int64_t first = ((blockIdx.x - a.token_ctas) * (kThreads / 32) + warp) * 32;
    const bool empty = first + lane < f.table_rows && __ldg(a.row_token + first + lane) < 0;
    uint32_t todo = __ballot_sync(0xffffffffu, empty);
    for (; todo; todo &= todo - 1) {
      T* at = drows + (first + __ffs(todo) - 1) * a.drows_stride;
      const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      for (int c = lane * W; c < f.hidden; c += 32 * W) {
        if constexpr (VEC)
          store8(at + c, zero);
        else
          at[c] = T(0);
      }
    }
    return;
  }
  __shared__ float part[kThreads / 32][kSlots];
  const int group = warp / a.warps, in_group = warp % a.warps;
  const int64_t t = int64_t(blockIdx.x) * ((kThreads / 32) / a.warps) + group;
  const bool live = t < f.tokens;
  const O* dy = static_cast<const O*>(a.dy) + t * a.dy_stride;
  for (int s0 = 0; s0 < f.top_k; s0 += kSlots) {
    int32_t r[kSlots];
    float w[kSlots], dot[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      const int s = s0 + j;
      r[j] = -1;
      w[j] = 1.0f;
      dot[j] = 0.0f;
      if (live && s < f.top_k) {
        r[j] = row_of(__ldg(f.token_row + t * f.top_k + s), f.table_rows, f.status);
        if (f.weights) w[j] = __ldg(f.weights + t * f.top_k + s);
        // (a row that another token holds is not this one's to write)
        if (r[j] >= 0 && __ldg(a.row_token + r[j]) != t) {
          atomicCAS(f.status, 0, int32_t(FO_ERR_ARG));
          r[j] = -1;
        }
      }
    }
    if (live)
      for (int c = (in_group * 32 + lane) * W; c < f.hidden; c += a.warps * 32 * W) {
        float g[W];
        if constexpr (VEC) {
          Pack8<O> p;
          p.load(dy + c);
          p.get(g);
          Pack8<T> v[kSlots];
          if (a.dweights) {
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
              if (r[j] >= 0) v[j].load_once(static_cast<const T*>(f.rows) + r[j] * f.row_stride + c);
          }
#pragma unroll
          for (int j = 0; j < kSlots; ++j)
            if (r[j] >= 0) {
              float x[8], d[8];
              if (a.dweights) {
                v[j].get(x);
#pragma unroll
                for (int i = 0; i < 8; ++i) dot[j] = fmaf(g[i], x[i], dot[j]);
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) d[i] = w[j] * g[i];
              store8(drows + r[j] * a.drows_stride + c, d);
            }
        } else {
          g[0] = widen(__ldg(dy + c));
#pragma unroll
          for (int j = 0; j < kSlots; ++j)
            if (r[j] >= 0) {
              if (a.dweights)
                dot[j] = fmaf(g[0], widen(__ldcs(static_cast<const T*>(f.rows) +
                                                 r[j] * f.row_stride + c)),
                              dot[j]);
              drows[r[j] * a.drows_stride + c] = narrow<T>(w[j] * g[0]);
            }
        }
      }
    if (!a.dweights) continue;
#pragma unroll
    for (int j = 0; j < kSlots; ++j) dot[j] = warp_sum(dot[j]);
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < kSlots; ++j) part[warp][j] = dot[j];
    }
    __syncthreads();
    if (in_group == 0 && lane < kSlots && live && s0 + lane < f.top_k) {
      float sum = 0.0f;
      for (int i = 0; i < a.warps; ++i) sum += part[warp + i][lane];
      a.dweights[t * f.top_k + s0 + lane] = sum;
    }
    __syncthreads();
  }
}

// 16-byte rows of 8-element pieces.
bool vec_rows(const void* p, int64_t stride, fo_type type) {
  const int64_t size = type == FO_TYPE_BF16 ? 2 : 4;
  return ((reinterpret_cast<uintptr_t>(p) | uintptr_t(stride * size)) & 15) == 0;
}

template <typename T, typename O>
void forward(const CombineArgs& a, bool vec, unsigned grid, cudaStream_t st) {
  if (vec)
    combine_kernel<T, O, true><<<grid, kThreads, 0, st>>>(a);
  else
    combine_kernel<T, O, false><<<grid, kThreads, 0, st>>>(a);
}

template <typename T, typename O>
void backward(const CombineBackArgs& a, bool vec, unsigned grid, cudaStream_t st) {
  if (vec)
    combine_backward_kernel<T, O, true><<<grid, kThreads, 0, st>>>(a);
  else
    combine_backward_kernel<T, O, false><<<grid, kThreads, 0, st>>>(a);
}

fo_status launched() { return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA; }

}  // namespace

fo_status launch_combine(const void* rows, fo_type type, int64_t table_rows, int64_t hidden,
                         int64_t row_stride, const int32_t* token_row, const float* weights,
                         int64_t tokens, int32_t top_k, void* y, fo_type y_type,
                         int64_t y_stride, int32_t* dev_status, void* stream) {
  CombineArgs a{};
  a.rows = rows, a.row_stride = row_stride, a.table_rows = table_rows;
  a.token_row = token_row, a.weights = weights;
  a.tokens = tokens, a.hidden = int32_t(hidden), a.top_k = top_k;
  a.y = y, a.y_stride = y_stride, a.status = dev_status;
  const bool vec = hidden % 8 == 0 && vec_rows(rows, row_stride, type) &&
                   vec_rows(y, y_stride, y_type);
  const int64_t chunks = vec ? hidden / 8 : hidden;
  a.pieces = int32_t((chunks + kThreads - 1) / kThreads);
  a.chunks = int32_t(chunks < kThreads ? chunks : kThreads);
  a.per_cta = a.pieces > 1 ? 1 : kThreads / a.chunks;
  const int64_t grid = (tokens + a.per_cta - 1) / a.per_cta * a.pieces;
  if (grid >= (int64_t(1) << 31)) return FO_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = type == FO_TYPE_BF16, ybf = y_type == FO_TYPE_BF16;
  if (bf && ybf)
    forward<uint16_t, uint16_t>(a, vec, unsigned(grid), st);
  else if (bf)
    forward<uint16_t, float>(a, vec, unsigned(grid), st);
  else if (ybf)
    forward<float, uint16_t>(a, vec, unsigned(grid), st);
  else
    forward<float, float>(a, vec, unsigned(grid), st);
  return launched();
}

fo_status launch_combine_backward(const void* dy, fo_type dy_type, int64_t dy_stride,
                                  const void* rows, fo_type type, int64_t table_rows,
                                  int64_t hidden, int64_t row_stride, const int32_t* token_row,
                                  const int32_t* row_token, const float* weights,
                                  int64_t tokens, int32_t top_k, void* drows,
                                  int64_t drows_stride, float* dweights, int32_t* dev_status,
                                  void* stream) {
  CombineBackArgs a{};
  CombineArgs& f = a.f;
  f.rows = rows, f.row_stride = row_stride, f.table_rows = table_rows;
  f.token_row = token_row, f.weights = weights;
  f.tokens = tokens, f.hidden = int32_t(hidden), f.top_k = top_k;
  f.status = dev_status;
  a.dy = dy, a.dy_stride = dy_stride, a.row_token = row_token;
  a.drows = drows, a.drows_stride = drows_stride, a.dweights = dweights;
  const bool vec = hidden % 8 == 0 && (!dweights || vec_rows(rows, row_stride, type)) &&
                   vec_rows(dy, dy_stride, dy_type) && vec_rows(drows, drows_stride, type);
  const int64_t warps = ((vec ? hidden / 8 : hidden) + 31) / 32;
  a.warps = warps <= 1 ? 1 : warps <= 2 ? 2 : warps <= 4 ? 4 : 8;
  const int64_t per_cta = (kThreads / 32) / a.warps;
  a.token_ctas = (tokens + per_cta - 1) / per_cta;
  const int64_t grid = a.token_ctas + (table_rows + kThreads - 1) / kThreads;
  if (grid == 0) return FO_OK;
  if (grid >= (int64_t(1) << 31)) return FO_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = type == FO_TYPE_BF16, ybf = dy_type == FO_TYPE_BF16;
  if (bf && ybf)
    backward<uint16_t, uint16_t>(a, vec, unsigned(grid), st);
  else if (bf)
    backward<uint16_t, float>(a, vec, unsigned(grid), st);
  else if (ybf)
    backward<float, uint16_t>(a, vec, unsigned(grid), st);
  else
    backward<float, float>(a, vec, unsigned(grid), st);
  return launched();
}

}  // namespace fo
