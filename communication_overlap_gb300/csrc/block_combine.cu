// The weighted sum of a token's rows of the experts' outputs, and its gradients.
//
//   y_t = sum over slots s of w_ts rows[r_ts],  r = token_row (-1: no row)
//   drows[r_ts] = w_ts dy_t,  dw_ts = <dy_t, rows[r_ts]>,  drows = 0 elsewhere.
//
// Both move each byte once and HBM bounds them.  Sums are fp32, in slot order;
// outputs are rounded once.
#include <cuda_runtime.h>

#include <mutex>

#include "block_common.cuh"

namespace fo {

namespace {

constexpr int kThreads = 256;

struct CombineArgs {
  const void* rows;
  int64_t row_stride, table_rows;
  const int32_t* token_row;
  const float* weights;    // NULL: ones
  int32_t tokens, hidden, top_k;
  void* y;
  int64_t y_stride;
  int32_t* status;
  // the shape of the work: an item is `per_item` tokens' columns of one piece
  int32_t pieces;          // items along a token's columns
  int32_t per_item;
  int32_t chunks;          // threads along a token's columns
  int32_t items;
};

// The row of a pair, -1 for none; a row outside the table is recorded.
__device__ __forceinline__ int row_of(int32_t r, int64_t table_rows, int32_t* status) {
  if (r < table_rows) return r;
  atomicCAS(status, 0, int32_t(FO_ERR_ARG));
  return -1;
}

// W columns of a row, as they lie in memory: eight on 16 bytes, or one.
template <typename T, int W>
struct Columns {
  Pack8<T> p;
  __device__ __forceinline__ void load_once(const T* at) { p.load_once(at); }
  __device__ __forceinline__ void load(const T* at) { p.load(at); }
  __device__ __forceinline__ void get(float (&v)[8]) const { p.get(v); }
  __device__ __forceinline__ static void store(T* at, const float (&v)[8]) { store8(at, v); }
};
template <typename T>
struct Columns<T, 1> {
  T e;
  __device__ __forceinline__ void load_once(const T* at) { e = __ldcs(at); }
  __device__ __forceinline__ void load(const T* at) { e = __ldg(at); }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = widen(e); }
  __device__ __forceinline__ static void store(T* at, const float (&v)[1]) {
    __stcs(at, narrow<T>(v[0]));
  }
};

// A thread takes W columns of TOKENS tokens, SLOTS of their slots at a time.  CTAs walk
// over the items, and the next item's rows are looked up while this one's are on
// their way: a look-up and the rows it names are two waits in a row otherwise.
template <typename T, typename O, int W, int SLOTS, int TOKENS>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs a) {
  const int local = a.pieces > 1 ? 0 : int(threadIdx.x) / a.chunks;
  const int lane_col = a.pieces > 1 ? int(threadIdx.x) : int(threadIdx.x) % a.chunks;
  const int per = a.per_item / TOKENS;      // from one of the thread's tokens to the next
  int32_t r[TOKENS][SLOTS];
  float w[TOKENS][SLOTS];
  const auto token = [&](int item, int i) {
    return int64_t(item / a.pieces) * a.per_item + local + i * per;
  };
  const auto column = [&](int item) {
    return (int64_t(item % a.pieces) * kThreads + lane_col) * W;
  };
  const auto look_up = [&](int item, int s0) {
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
      const int64_t t = token(item, i);
      const bool live = item < a.items && local < per && t < a.tokens;
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) {
        const bool has = live && s0 + j < a.top_k;
        r[i][j] = has ? __ldg(a.token_row + t * a.top_k + s0 + j) : -1;
        w[i][j] = has && a.weights ? __ldg(a.weights + t * a.top_k + s0 + j) : 1.0f;
      }
    }
  };
  look_up(blockIdx.x, 0);
  for (int item = blockIdx.x; item < a.items; item += gridDim.x) {
    const int64_t col = column(item);
    const bool in = col < a.hidden;
    const T* rows = static_cast<const T*>(a.rows) + col;
    float acc[TOKENS][W];
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
#pragma unroll
      for (int k = 0; k < W; ++k) acc[i][k] = 0.0f;
    }
    for (int s0 = 0; s0 < a.top_k; s0 += SLOTS) {
      Columns<T, W> v[TOKENS][SLOTS];
      float by[TOKENS][SLOTS];
      bool has[TOKENS][SLOTS];
#pragma unroll
      for (int i = 0; i < TOKENS; ++i) {
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
          const int row = r[i][j] < 0 ? -1 : row_of(r[i][j], a.table_rows, a.status);
          has[i][j] = in && row >= 0;
          by[i][j] = w[i][j];
          if (has[i][j]) v[i][j].load_once(rows + row * a.row_stride);
        }
      }
      if (s0 + SLOTS < a.top_k)
        look_up(item, s0 + SLOTS);
      else
        look_up(item + gridDim.x, 0);
#pragma unroll
      for (int i = 0; i < TOKENS; ++i) {
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
          if (has[i][j]) {
            float f[W];
            v[i][j].get(f);
#pragma unroll
            for (int k = 0; k < W; ++k) acc[i][k] = fmaf(by[i][j], f[k], acc[i][k]);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
      const int64_t t = token(item, i);
      if (in && local < per && t < a.tokens)
        Columns<O, W>::store(static_cast<O*>(a.y) + t * a.y_stride + col, acc[i]);
    }
  }
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
};

// A token per group of warps, SLOTS of its slots at a time: dy, the rows, their
// products and the rows' gradients, CHUNKS times W columns per thread under way; then
// the products' sums over the group.  CTAs walk over the tokens; the rows of the next
// token are looked up, and checked against row_token, two tokens and one ahead.
template <typename T, typename O, int W, int SLOTS, int CHUNKS>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const CombineBackArgs a) {
  __shared__ float part[2][kThreads / 32][SLOTS];
  const CombineArgs& f = a.f;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / a.warps, in_group = warp % a.warps;
  const int per = (kThreads / 32) / a.warps;           // tokens of a CTA
  const int64_t step = int64_t(gridDim.x) * per;
  const T* rows = static_cast<const T*>(f.rows);
  T* drows = static_cast<T*>(a.drows);
  int turn = 0;
  // the first slots of a token: its rows, and the tokens that those name
  const auto look_up = [&](int64_t t, int s0, int32_t (&r)[SLOTS], float (&w)[SLOTS]) {
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      const bool has = t < f.tokens && s0 + j < f.top_k;
      r[j] = has ? __ldg(f.token_row + t * f.top_k + s0 + j) : -1;
      w[j] = has && f.weights ? __ldg(f.weights + t * f.top_k + s0 + j) : 1.0f;
    }
  };
  const auto named = [&](const int32_t (&r)[SLOTS], int32_t (&by)[SLOTS]) {
#pragma unroll
    for (int j = 0; j < SLOTS; ++j)
      by[j] = r[j] >= 0 && r[j] < f.table_rows ? __ldg(a.row_token + r[j]) : -1;
  };
  const int64_t first = int64_t(blockIdx.x) * per + group;
  int32_t r[SLOTS], by[SLOTS], next_r[SLOTS];
  float w[SLOTS], next_w[SLOTS];
  look_up(first, 0, r, w);
  named(r, by);
  look_up(first + step, 0, next_r, next_w);
  // (as many rounds for all of the CTA's groups: they meet at the sums)
  for (int64_t base = int64_t(blockIdx.x) * per; base < f.tokens; base += step) {
    const int64_t t = base + group;
    const bool live = t < f.tokens;
    const O* dy = static_cast<const O*>(a.dy) + t * a.dy_stride;
    int32_t next_by[SLOTS], then_r[SLOTS];
    float then_w[SLOTS];
    named(next_r, next_by);
    look_up(t + 2 * step, 0, then_r, then_w);
    for (int s0 = 0; s0 < f.top_k; s0 += SLOTS) {
      if (s0 > 0) {
        look_up(t, s0, r, w);
        named(r, by);
      }
      float dot[SLOTS];
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) {
        dot[j] = 0.0f;
        // (a row outside the table, or one that holds another token, is not this one's)
        if (live && r[j] >= 0 && by[j] != int32_t(t)) {
          atomicCAS(f.status, 0, int32_t(FO_ERR_ARG));
          r[j] = -1;
        }
      }
      const int stride = a.warps * 32 * W;
      if (live)
        for (int c0 = (in_group * 32 + lane) * W; c0 < f.hidden; c0 += CHUNKS * stride) {
          Columns<O, W> g[CHUNKS];
          Columns<T, W> v[CHUNKS][SLOTS];
#pragma unroll
          for (int k = 0; k < CHUNKS; ++k) {
            const int c = c0 + k * stride;
            if (c >= f.hidden) continue;
            if (f.top_k > SLOTS)
              g[k].load(dy + c);
            else
              g[k].load_once(dy + c);
            if (a.dweights) {
#pragma unroll
              for (int j = 0; j < SLOTS; ++j)
                if (r[j] >= 0) v[k][j].load_once(rows + r[j] * f.row_stride + c);
            }
          }
#pragma unroll
          for (int k = 0; k < CHUNKS; ++k) {
            const int c = c0 + k * stride;
            if (c >= f.hidden) continue;
            float x[W];
            g[k].get(x);
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
              if (r[j] >= 0) {
                float y[W];
                if (a.dweights) {
                  v[k][j].get(y);
#pragma unroll
                  for (int i = 0; i < W; ++i) dot[j] = fmaf(x[i], y[i], dot[j]);
                }
#pragma unroll
                for (int i = 0; i < W; ++i) y[i] = w[j] * x[i];
                Columns<T, W>::store(drows + r[j] * a.drows_stride + c, y);
              }
          }
        }
      if (!a.dweights) continue;
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) dot[j] = warp_sum(dot[j]);
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) part[turn][warp][j] = dot[j];
      }
      __syncthreads();
      if (in_group == 0 && lane < SLOTS && live && s0 + lane < f.top_k) {
        float sum = 0.0f;
        for (int i = 0; i < a.warps; ++i) sum += part[turn][warp + i][lane];
        a.dweights[t * f.top_k + s0 + lane] = sum;
      }
      turn ^= 1;
    }
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      r[j] = next_r[j], w[j] = next_w[j], by[j] = next_by[j];
      next_r[j] = then_r[j], next_w[j] = then_w[j];
    }
  }
  // the rows that hold no token become zeros: 32 of them looked at by a warp
  const int64_t looks = (f.table_rows + 31) / 32;
  for (int64_t i = int64_t(blockIdx.x) * (kThreads / 32) + warp; i < looks;
       i += int64_t(gridDim.x) * (kThreads / 32)) {
    const int64_t row = i * 32 + lane;
    uint32_t todo = __ballot_sync(0xffffffffu, row < f.table_rows && __ldg(a.row_token + row) < 0);
    for (; todo; todo &= todo - 1) {
      T* at = drows + (i * 32 + __ffs(todo) - 1) * a.drows_stride;
      float zero[W];
#pragma unroll
      for (int k = 0; k < W; ++k) zero[k] = 0.0f;
      for (int c = lane * W; c < f.hidden; c += 32 * W) Columns<T, W>::store(at + c, zero);
    }
  }
}

// 16-byte rows of 8-element pieces.
bool vec_rows(const void* p, int64_t stride, fo_type type) {
  const int64_t size = type == FO_TYPE_BF16 ? 2 : 4;
  return ((reinterpret_cast<uintptr_t>(p) | uintptr_t(stride * size)) & 15) == 0;
}

// How many CTAs of a kernel the device holds at once, asked for once per device.
template <auto K>
fo_status resident(int* ctas) {
  static std::once_flag once[64];
  static int count[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FO_ERR_CUDA;
  const int slot = dev < 64 ? dev : 63;
  std::call_once(once[slot], [&] {
    int per_sm = 0, sms = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, K, kThreads, 0) == cudaSuccess &&
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
      count[slot] = per_sm * sms;
  });
  *ctas = count[slot];
  return count[slot] > 0 ? FO_OK : FO_ERR_CUDA;
}

template <typename T, typename O, int W, int SLOTS, int TOKENS>
fo_status forward_as(CombineArgs a, cudaStream_t st) {
  const int64_t chunks = (a.hidden + W - 1) / W;
  a.pieces = int32_t((chunks + kThreads - 1) / kThreads);
  a.chunks = int32_t(chunks < kThreads ? chunks : kThreads);
  a.per_item = (a.pieces > 1 ? 1 : kThreads / a.chunks) * TOKENS;
  const int64_t items = (int64_t(a.tokens) + a.per_item - 1) / a.per_item * a.pieces;
  if (items >= (int64_t(1) << 30)) return FO_ERR_UNSUPPORTED;
  a.items = int32_t(items);
  constexpr auto kernel = combine_kernel<T, O, W, SLOTS, TOKENS>;
  int ctas = 0;
  const fo_status q = resident<kernel>(&ctas);
  if (q != FO_OK) return q;
  kernel<<<unsigned(items < ctas ? items : ctas), kThreads, 0, st>>>(a);
  return FO_OK;
}

template <typename T, typename O>
fo_status forward(const CombineArgs& a, bool vec, cudaStream_t st) {
  if (!vec) return forward_as<T, O, 1, 4, 2>(a, st);
  if (a.top_k <= 2) return forward_as<T, O, 8, 2, 2>(a, st);
  return forward_as<T, O, 8, 4, 1>(a, st);
}

template <typename T, typename O, int W, int SLOTS, int CHUNKS>
fo_status backward_as(const CombineBackArgs& a, cudaStream_t st) {
  const int64_t per = (kThreads / 32) / a.warps;
  int64_t grid = (int64_t(a.f.tokens) + per - 1) / per;
  const int64_t looks = (a.f.table_rows + kThreads - 1) / kThreads;
  if (grid < looks) grid = looks;
  constexpr auto kernel = combine_backward_kernel<T, O, W, SLOTS, CHUNKS>;
  int ctas = 0;
  const fo_status q = resident<kernel>(&ctas);
  if (q != FO_OK) return q;
  kernel<<<unsigned(grid < ctas ? grid : ctas), kThreads, 0, st>>>(a);
  return FO_OK;
}

template <typename T, typename O>
fo_status backward(const CombineBackArgs& a, bool vec, cudaStream_t st) {
  if (!vec) return backward_as<T, O, 1, 4, 2>(a, st);
  if (a.f.top_k <= 2) return backward_as<T, O, 8, 2, 2>(a, st);
  return backward_as<T, O, 8, 4, 1>(a, st);
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
  a.tokens = int32_t(tokens), a.hidden = int32_t(hidden), a.top_k = top_k;
  a.y = y, a.y_stride = y_stride, a.status = dev_status;
  const bool vec = hidden % 8 == 0 && vec_rows(rows, row_stride, type) &&
                   vec_rows(y, y_stride, y_type);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = type == FO_TYPE_BF16, ybf = y_type == FO_TYPE_BF16;
  const fo_status q = bf && ybf ? forward<uint16_t, uint16_t>(a, vec, st)
                      : bf      ? forward<uint16_t, float>(a, vec, st)
                      : ybf     ? forward<float, uint16_t>(a, vec, st)
                                : forward<float, float>(a, vec, st);
  return q == FO_OK ? launched() : q;
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
  f.tokens = int32_t(tokens), f.hidden = int32_t(hidden), f.top_k = top_k;
  f.status = dev_status;
  a.dy = dy, a.dy_stride = dy_stride, a.row_token = row_token;
  a.drows = drows, a.drows_stride = drows_stride, a.dweights = dweights;
  const bool vec = hidden % 8 == 0 && (!dweights || vec_rows(rows, row_stride, type)) &&
                   vec_rows(dy, dy_stride, dy_type) && vec_rows(drows, drows_stride, type);
  const int64_t warps = ((vec ? hidden / 8 : hidden) + 31) / 32;
  a.warps = warps <= 1 ? 1 : warps <= 2 ? 2 : warps <= 4 ? 4 : 8;
  if (tokens == 0 && table_rows == 0) return FO_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = type == FO_TYPE_BF16, ybf = dy_type == FO_TYPE_BF16;
  const fo_status q = bf && ybf ? backward<uint16_t, uint16_t>(a, vec, st)
                      : bf      ? backward<uint16_t, float>(a, vec, st)
                      : ybf     ? backward<float, uint16_t>(a, vec, st)
                                : backward<float, float>(a, vec, st);
  return q == FO_OK ? launched() : q;
}

}  // namespace fo
