// Gradients of the norm (block_norm.cu).  With xn = x r1, u = xn post (x without
// post), q = scale gate, s = residual + q u, sn = s r2, means over a row:
//
//   D  = dsum + r2 (dy pre - sn mean(dy pre sn))            = dresidual
//   dx = r1 (q D post - xn mean(q D post xn))               (q D without post)
//   dpre = sum over tokens of dy sn,  dpost: of q D xn,
//   dgate: of scale u D, over the tokens that share the gate's row.
//
// The second mean needs D, hence the first.  It is linear in D, so both come
// from one round of sums over the row: with w = q post xn,
//   a = sum dy pre sn,  b = sum w (dsum + r2 dy pre),  c = sum w sn,
//   mean(q D post xn) = (b - r2 (a / H) c) / H.
// s is formed again from x and the residual, unrounded, instead of being read.
//
// A worker takes a contiguous range of tokens and keeps the parameters' sums of
// its columns in registers; a last kernel adds the workers' in their order, so
// results do not vary from run to run.  Rows of up to 4096 columns on 16 bytes go
// through one kernel, which holds a row in registers between the two passes;
// others through two, one for the means and one for the columns.
#include <cuda_runtime.h>

#include "block_norm.cuh"

namespace fo {

namespace {

constexpr int64_t kWorkers = 2048;      // the most

struct BackShape {
  int32_t workers, per_worker;
  float2* means;        // [tokens] where the rows take two kernels
  float* pre_part;      // [workers][hidden]
  float* post_part;     // [workers][hidden]
  float* gate_part;     // [workers + gates][hidden]: worker w's part of gate row b at w + b
};

// What a column of a token brings along.
template <typename A, typename S, int W>
struct Columns {
  Piece<A, W> px, py;
  Piece<S, W> pr, pd;

  __device__ __forceinline__ void load(const NormBackArgs& a, int64_t t, int col, bool live) {
    const NormArgs& f = a.f;
    px.load(static_cast<const A*>(f.x) + t * f.x_stride + col, live);
    py.load(static_cast<const A*>(a.dy) + t * a.dy_stride + col, live && f.pre != nullptr);
    pr.load(static_cast<const S*>(f.residual) + t * f.residual_stride + col,
            live && f.residual != nullptr);
    pd.load(static_cast<const S*>(a.dsum) + t * a.dsum_stride + col, live && a.dsum != nullptr);
  }
  // xn; u; q; w = q post; sn; dy; e = dy pre; d = dsum
  __device__ __forceinline__ void values(const NormBackArgs& a, int col, int64_t gate_row,
                                         float r1, float r2, float (&xn)[W], float (&u)[W],
                                         float (&q)[W], float (&w)[W], float (&sn)[W],
                                         float (&dy)[W], float (&e)[W], float (&d)[W]) const {
    const NormArgs& f = a.f;
    float p[W];
    px.get(xn);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      xn[i] *= r1;
      u[i] = xn[i];
      q[i] = f.scale;
      e[i] = 0.0f;
    }
    if (f.gate != nullptr) {
      load_param<W>(f.gate, gate_row + col, f.params_f32, p);
#pragma unroll
      for (int i = 0; i < W; ++i) q[i] *= p[i];
    }
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = q[i];
    if (f.post != nullptr) {
      load_param<W>(f.post, col, f.params_f32, p);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        u[i] *= p[i];
        w[i] *= p[i];
      }
    }
    pr.get(sn);
    py.get(dy);
    pd.get(d);
#pragma unroll
    for (int i = 0; i < W; ++i) sn[i] = fmaf(q[i], u[i], sn[i]) * r2;
    if (f.pre != nullptr) {
      load_param<W>(f.pre, col, f.params_f32, p);
#pragma unroll
      for (int i = 0; i < W; ++i) e[i] = dy[i] * p[i];
    }
  }
  // The three sums' share of these columns.
  __device__ __forceinline__ void sums(const NormBackArgs& a, int col, int64_t gate_row, float r1,
                                       float r2, float (&sum)[3]) const {
    float xn[W], u[W], q[W], w[W], sn[W], dy[W], e[W], d[W];
    values(a, col, gate_row, r1, r2, xn, u, q, w, sn, dy, e, d);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float wx = w[i] * xn[i];
      sum[0] = fmaf(e[i], sn[i], sum[0]);
      sum[1] = fmaf(wx, fmaf(r2, e[i], d[i]), sum[1]);
      sum[2] = fmaf(wx, sn[i], sum[2]);
    }
  }
  // Gradients of these columns, and their share of the parameters'.
  __device__ __forceinline__ void gradients(const NormBackArgs& a, int64_t t, int col,
                                            int64_t gate_row, float r1, float r2, float m1,
                                            float m2, float (&dpre)[W], float (&dpost)[W],
                                            float (&dgate)[W]) const {
    const NormArgs& f = a.f;
    float xn[W], u[W], q[W], w[W], sn[W], dy[W], e[W], d[W];
    values(a, col, gate_row, r1, r2, xn, u, q, w, sn, dy, e, d);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      d[i] += r2 * (e[i] - sn[i] * m2);
      dpre[i] = fmaf(dy[i], sn[i], dpre[i]);
      dgate[i] = fmaf(f.scale * u[i], d[i], dgate[i]);
      dpost[i] = fmaf(q[i] * d[i], xn[i], dpost[i]);
      e[i] = w[i] * d[i];
      if (f.post != nullptr) e[i] = r1 * (e[i] - xn[i] * m1);
    }
    if (a.dresidual != nullptr)
      store_piece<W>(static_cast<S*>(a.dresidual) + t * a.dresidual_stride + col, d);
    store_piece<W>(static_cast<A*>(a.dx) + t * a.dx_stride + col, e);
  }
};

__device__ __forceinline__ void means_of(const float (&sum)[3], float r2, int hidden, float& m1,
                                         float& m2) {
  m2 = sum[0] / float(hidden);
  m1 = (sum[1] - r2 * m2 * sum[2]) / float(hidden);
}

// The gate's sums of W columns, where a token is the last of its gate's row or of
// the worker's.
template <int W>
__device__ __forceinline__ void flush_gate(const NormBackArgs& a, const BackShape& n, int64_t t,
                                           int64_t t1, int64_t worker, int col,
                                           float (&dgate)[W]) {
  const NormArgs& f = a.f;
  if (f.gate == nullptr || (t + 1 != t1 && (t + 1) % f.gate_rows != 0)) return;
  if (f.gate_rows > 1)
    store_piece<W>(n.gate_part + (worker + t / f.gate_rows) * f.hidden + col, dgate);
  else if (f.params_f32)
    store_piece<W>(static_cast<float*>(a.dgate) + t * f.hidden + col, dgate);
  else
    store_piece<W>(static_cast<uint16_t*>(a.dgate) + t * f.hidden + col, dgate);
#pragma unroll
  for (int i = 0; i < W; ++i) dgate[i] = 0.0f;
}

template <int W>
__device__ __forceinline__ void store_parts(const NormBackArgs& a, const BackShape& n,
                                            int64_t worker, int col, const float (&dpre)[W],
                                            const float (&dpost)[W]) {
  const NormArgs& f = a.f;
  if (f.pre != nullptr) store_piece<W>(n.pre_part + worker * f.hidden + col, dpre);
  if (f.post != nullptr) store_piece<W>(n.post_part + worker * f.hidden + col, dpost);
}

// A worker per row of threads, eight columns per thread; several to a CTA where a
// row has up to four warps.
template <typename A, typename S>
__global__ void __launch_bounds__(512) norm_backward_kernel(const NormBackArgs a,
                                                            const BackShape n, int warps) {
  __shared__ float buf[2 * 3 * 32];
  int turn = 0;
  const NormArgs& f = a.f;
  const int row = int(threadIdx.x >> 5) / warps;
  const int col = (int(threadIdx.x) - row * warps * 32) * 8;
  const int64_t worker = int64_t(blockIdx.x) * (int(blockDim.x) / (warps * 32)) + row;
  const int64_t t0 = worker * n.per_worker;
  const int64_t t1 = min(t0 + n.per_worker, int64_t(f.tokens));
  float dpre[8], dpost[8], dgate[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dpre[i] = dpost[i] = dgate[i] = 0.0f;
  Columns<A, S, 8> next;
  next.load(a, t0, col, t0 < t1 && col < f.hidden);
  // (the same number of rounds for all of the CTA: they meet at the sums)
  for (int k = 0; k < n.per_worker; ++k) {
    const int64_t t = t0 + k;
    const bool live = t < t1 && col < f.hidden;
    const Columns<A, S, 8> c = next;
    next.load(a, t + 1, col, t + 1 < t1 && col < f.hidden);
    const float r1 = live && f.post ? f.post_rstd[t] : 1.0f;
    const float r2 = live && f.pre ? f.pre_rstd[t] : 0.0f;
    const int64_t gate_row = live && f.gate ? t / f.gate_rows * f.gate_stride : 0;
    float sum[3] = {0.0f, 0.0f, 0.0f};
    if (live) c.sums(a, col, gate_row, r1, r2, sum);
    row_sums<3>(sum, row * warps, warps, buf, turn);
    if (!live) continue;
    float m1, m2;
    means_of(sum, r2, f.hidden, m1, m2);
    c.gradients(a, t, col, gate_row, r1, r2, m1, m2, dpre, dpost, dgate);
    flush_gate<8>(a, n, t, t1, worker, col, dgate);
  }
  if (t0 < t1 && col < f.hidden) store_parts<8>(a, n, worker, col, dpre, dpost);
}

// Any rows, first: the two means of each token, by a CTA.
template <typename A, typename S, int W>
__global__ void __launch_bounds__(512) norm_means_kernel(const NormBackArgs a, const BackShape n) {
  __shared__ float buf[2 * 3 * 32];
  int turn = 0;
  const NormArgs& f = a.f;
  const int64_t t = blockIdx.x;
  const float r1 = f.post ? f.post_rstd[t] : 1.0f;
  const float r2 = f.pre ? f.pre_rstd[t] : 0.0f;
  const int64_t gate_row = f.gate ? t / f.gate_rows * f.gate_stride : 0;
  float sum[3] = {0.0f, 0.0f, 0.0f};
  for (int col = int(threadIdx.x) * W; col < f.hidden; col += int(blockDim.x) * W) {
    Columns<A, S, W> c;
    c.load(a, t, col, true);
    c.sums(a, col, gate_row, r1, r2, sum);
  }
  row_sums<3>(sum, 0, int(blockDim.x) >> 5, buf, turn);
  float m1, m2;
  means_of(sum, r2, f.hidden, m1, m2);
  if (threadIdx.x == 0) n.means[t] = make_float2(m1, m2);
}

// Then the columns: a CTA takes 256 threads' columns of a worker's tokens.
template <typename A, typename S, int W>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormBackArgs a,
                                                           const BackShape n, int pieces) {
  const NormArgs& f = a.f;
  const int64_t worker = blockIdx.x / unsigned(pieces);
  const int col = (int(blockIdx.x % unsigned(pieces)) * 256 + int(threadIdx.x)) * W;
  if (col >= f.hidden) return;
  const int64_t t0 = worker * n.per_worker;
  const int64_t t1 = min(t0 + n.per_worker, int64_t(f.tokens));
  float dpre[W], dpost[W], dgate[W];
#pragma unroll
  for (int i = 0; i < W; ++i) dpre[i] = dpost[i] = dgate[i] = 0.0f;
  Columns<A, S, W> next;
  next.load(a, t0, col, t0 < t1);
  for (int64_t t = t0; t < t1; ++t) {
    const Columns<A, S, W> c = next;
    next.load(a, t + 1, col, t + 1 < t1);
    const float2 m = n.means[t];
    c.gradients(a, t, col, f.gate ? t / f.gate_rows * f.gate_stride : 0,
                f.post ? f.post_rstd[t] : 1.0f, f.pre ? f.pre_rstd[t] : 0.0f, m.x, m.y, dpre,
                dpost, dgate);
    flush_gate<W>(a, n, t, t1, worker, col, dgate);
  }
  store_parts<W>(a, n, worker, col, dpre, dpost);
}

// The parts' sums: a CTA takes 32 columns of one result, its warps every eighth
// part, and joins them in their order.
__global__ void __launch_bounds__(256) norm_join_kernel(const NormBackArgs a, const BackShape n,
                                                        int columns) {
  __shared__ float buf[8][33];
  const NormArgs& f = a.f;
  int64_t which = blockIdx.x / unsigned(columns);
  const int col = int(blockIdx.x % unsigned(columns)) * 32 + (threadIdx.x & 31);
  const int warp = threadIdx.x >> 5;
  const float* from = nullptr;
  void* to = nullptr;
  int64_t lo = 0, hi = n.workers, at = 0;
  if (f.pre != nullptr && which-- == 0) {
    from = n.pre_part, to = a.dpre;
  } else if (f.post != nullptr && which-- == 0) {
    from = n.post_part, to = a.dpost;
  } else {
    // the workers whose tokens meet gate row `which`
    from = n.gate_part + which * f.hidden, to = a.dgate;
    at = which * f.hidden;
    const int64_t first = which * f.gate_rows;
    lo = n.workers ? first / n.per_worker : 0;
    hi = n.workers ? (first + f.gate_rows - 1) / n.per_worker + 1 : 0;
  }
  float sum = 0.0f;
  if (col < f.hidden) {
#pragma unroll 4
    for (int64_t w = lo + warp; w < hi; w += 8) sum += __ldcs(from + w * f.hidden + col);
  }
  buf[warp][threadIdx.x & 31] = sum;
  __syncthreads();
  if (warp != 0 || col >= f.hidden) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) sum += buf[i][threadIdx.x];
  if (f.params_f32)
    static_cast<float*>(to)[at + col] = sum;
  else
    static_cast<uint16_t*>(to)[at + col] = narrow<uint16_t>(sum);
}

// Workers of at least as many as are asked for, where there are the tokens.
void share_out(BackShape* n, int64_t tokens, int64_t most) {
  if (most > kWorkers) most = kWorkers;
  n->per_worker = int32_t((tokens + most - 1) / most);
  n->workers = int32_t((tokens + n->per_worker - 1) / n->per_worker);
}

template <typename A, typename S>
void launch(const NormBackArgs& a, BackShape* n, float* workspace, bool vec, int sms,
            cudaStream_t st) {
  const NormArgs& f = a.f;
  const int64_t H = f.hidden;
  const bool whole = vec && H <= 4096;
  const int warps = int((H + 255) / 256), rows = warps <= 4 ? 8 / warps : 1;
  const int width = vec ? 8 : 1;
  const int64_t pieces = (H + 256 * width - 1) / (256 * width);
  if (whole) {
    share_out(n, f.tokens, int64_t(sms) * rows);
  } else {
    share_out(n, f.tokens, (int64_t(sms) * 4 + pieces - 1) / pieces);
    n->means = reinterpret_cast<float2*>(workspace);
    workspace += (2 * int64_t(f.tokens) + 3) / 4 * 4;
  }
  n->pre_part = workspace;
  n->post_part = n->pre_part + n->workers * H;
  n->gate_part = n->post_part + n->workers * H;
  if (whole) {
    norm_backward_kernel<A, S><<<unsigned((n->workers + rows - 1) / rows), rows * warps * 32, 0, st>>>(
        a, *n, warps);
    return;
  }
  const unsigned grid = unsigned(n->workers * pieces);
  if (vec) {
    norm_means_kernel<A, S, 8><<<unsigned(f.tokens), 512, 0, st>>>(a, *n);
    norm_columns_kernel<A, S, 8><<<grid, 256, 0, st>>>(a, *n, int(pieces));
  } else {
    const int w = int((H + 31) / 32);
    norm_means_kernel<A, S, 1><<<unsigned(f.tokens), (w < 16 ? w : 16) * 32, 0, st>>>(a, *n);
    norm_columns_kernel<A, S, 1><<<grid, 256, 0, st>>>(a, *n, int(pieces));
  }
}

}  // namespace

// Both means of every token, and the workers' parts (a multiple of 16 bytes each
// where the rows are).
int64_t block_norm_workspace_bytes(int64_t tokens, int64_t hidden, int64_t gates) {
  const int64_t workers = tokens < kWorkers ? tokens : kWorkers;
  const int64_t gate_parts = gates > 0 && gates < tokens ? workers + gates : 0;
  return 8 * tokens + 16 + 4 * hidden * (2 * workers + gate_parts);
}

fo_status launch_block_norm_backward(const NormBackArgs& a, fo_type type, fo_type stream_type,
                                     int64_t gates, void* stream) {
  const NormArgs& f = a.f;
  const int64_t sa = size_of(type), ss = size_of(stream_type), sp = f.params_f32 ? 4 : 2;
  const bool vec = norm_rows_on_16(f, type, stream_type) && norm_on_16(a.dsum, a.dsum_stride, ss) &&
                   norm_on_16(a.dy, a.dy_stride, sa) && norm_on_16(a.dx, a.dx_stride, sa) &&
                   norm_on_16(a.dresidual, a.dresidual_stride, ss) &&
                   norm_on_16(a.dgate, f.hidden, sp);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FO_ERR_CUDA;
  // (a gate's row for every token is written by the kernel itself)
  const int64_t joined = f.gate && f.gate_rows != 1 ? gates : 0;
  const int64_t results = (f.pre != nullptr) + (f.post != nullptr) + joined;
  const int64_t columns = (f.hidden + 31) / 32;
  if (results * columns >= (int64_t(1) << 31)) return FO_ERR_UNSUPPORTED;
  BackShape n{};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // (without tokens there are no parts, and the sums are zeros)
  if (f.tokens > 0) {
    if (type == FO_TYPE_F32)
      launch<float, float>(a, &n, a.workspace, vec, sms, st);
    else if (stream_type == FO_TYPE_F32)
      launch<uint16_t, float>(a, &n, a.workspace, vec, sms, st);
    else
      launch<uint16_t, uint16_t>(a, &n, a.workspace, vec, sms, st);
  }
  if (cudaGetLastError() != cudaSuccess) return FO_ERR_CUDA;
  if (results > 0)
    norm_join_kernel<<<unsigned(results * columns), 256, 0, st>>>(a, n, int(columns));
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace fo
