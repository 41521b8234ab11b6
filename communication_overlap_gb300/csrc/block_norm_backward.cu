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
// s is formed again from x and the residual, unrounded, instead of being read.  Without
// pre D = dsum, and no value of s enters: an infinity or a NaN of it must not by way of
// r2 = 0 either, so kernels that hold a row have that form by itself (PRE).
//
// A worker takes a contiguous range of tokens and keeps the parameters' sums of
// its columns in registers; a last kernel adds the workers' in their order, so
// results do not vary from run to run.  Rows on 16 bytes of up to 8192 columns (of bf16
// into an fp32 stream 6656, of fp32 5632: two rows and the parameters have to fit in
// shared memory), and others of up to 4096, go through one kernel, which holds a row in
// registers between the two passes; the rest through two, one for the means and one for
// the columns.
//
// 16384 x 4096 of bf16: 805 MB in 130 us (6.2 TB/s) and 7 us for the joining kernel,
// whose launch most of that is; 4095 x 2752 of bf16 with an fp32 stream 203 MB in 42
// (4.8) and 7.  Rows of 8192 move 4.3 TB/s, 12288 in two kernels 2.4.  Without pre,
// 16384 x 4096 of bf16, 537 MB in 92 us (5.8).
#include <cuda_runtime.h>

#include "block_norm.cuh"

namespace fo {

namespace {

constexpr int kMaxSms = 192;      // that take part

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
    for (int i = 0; i < W; ++i)
      sn[i] = f.pre != nullptr ? fmaf(q[i], u[i], sn[i]) * r2 : 0.0f;
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

// A worker's sums for W columns of a gate's row, which token t is the last of here.
template <int W>
__device__ __forceinline__ void store_gate(const NormBackArgs& a, const BackShape& n, int64_t t,
                                           int64_t worker, int col, const float (&dgate)[W]) {
  const NormArgs& f = a.f;
  if (f.gate_rows > 1)
    store_piece<W>(n.gate_part + (worker + t / f.gate_rows) * f.hidden + col, dgate);
  else if (f.params_f32)
    store_piece<W>(static_cast<float*>(a.dgate) + t * f.hidden + col, dgate);
  else
    store_piece<W>(static_cast<uint16_t*>(a.dgate) + t * f.hidden + col, dgate);
}

// scale times eight values of a parameter from `i` on, or scale alone.
__device__ __forceinline__ void factor_of(const NormArgs& f, const void* p, int64_t i,
                                          float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = 1.0f;
  if (p != nullptr) load_param<8>(p, i, f.params_f32, v);
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= f.scale;
}

__device__ __forceinline__ void store_pairs(float* p, const Pair (&x)[4]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i].get(v[2 * i], v[2 * i + 1]);
  store8(p, v);
}

template <int W>
__device__ __forceinline__ void store_parts(const NormBackArgs& a, const BackShape& n,
                                            int64_t worker, int col, const float (&dpre)[W],
                                            const float (&dpost)[W]) {
  const NormArgs& f = a.f;
  if (f.pre != nullptr) store_piece<W>(n.pre_part + worker * f.hidden + col, dpre);
  if (f.post != nullptr) store_piece<W>(n.post_part + worker * f.hidden + col, dpost);
}

// Rows of up to 8192 columns; a worker per row of threads, several to a CTA where a
// row has few warps.  DEPTH rows are under way in the ring, the parameters' product w =
// scale gate post and pre lie behind it, and one instruction takes two values.  Of the
// parameters' sums two are kept: of dy sn, and G of xn D over tokens with the same
// gate, since dgate = scale post G and dpost = scale gate G (summed over the gates,
// where a worker meets several: GATES).  PRE: there is a norm before the next block.
// 16384 x 4096: eight columns per thread and one value per instruction took 174 us.
template <typename A, typename S, int NV, int DEPTH, bool GATES, bool PRE>
__global__ void __launch_bounds__(512, 1) norm_backward_kernel(const NormBackArgs a,
                                                               const BackShape n, int warps) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float buf[2 * 8 * 48];           // of up to eight rows
  constexpr int kA = sizeof(A) / 2, kS = sizeof(S) / 2;     // pieces of eight columns
  constexpr int kOf = 2 * (kA + kS);                        // x, dy, residual, dsum
  constexpr int kPieces = NV * kOf;
  // the parameters: in registers, or of two times eight columns in pieces of their own
  constexpr bool kKeep = NV == 1;
  constexpr int kW = DEPTH * kPieces, kPre = kW + 2 * NV;
  for (int i = threadIdx.x; i < 2 * 8 * 48; i += blockDim.x) buf[i] = 0.0f;
  __syncthreads();
  int turn = 0;
  const NormArgs& f = a.f;
  const RowGroup g = RowGroup::of(warps);
  const OwnRing ring(smem);
  // (asked at run time as well: 8192 columns 201 us, where PRE alone decides 214)
  const auto normed = [&] { return PRE && f.pre != nullptr; };
  int col[NV];
  bool has[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    // (threads without columns work on the zeros that the ring starts with)
    col[v] = (v * warps * 32 + g.tid) * 8;
    has[v] = col[v] < f.hidden;
  }
  const int64_t worker = int64_t(blockIdx.x) * (int(blockDim.x) / (warps * 32)) + g.index;
  const int t0 = int(min(worker * n.per_worker, int64_t(f.tokens)));
  const int t1 = min(t0 + n.per_worker, f.tokens);
  const float inv = 1.0f / float(f.hidden);
  const A* x_at = static_cast<const A*>(f.x) + t0 * f.x_stride;
  const A* dy_at = static_cast<const A*>(a.dy) + t0 * a.dy_stride;
  const S* r_at = static_cast<const S*>(f.residual) + t0 * f.residual_stride;
  const S* d_at = static_cast<const S*>(a.dsum) + t0 * a.dsum_stride;
  int fetched = t0;
  // (what is not given stays the zeros that the ring starts with)
  const auto fetch = [&](int stage) {
    if (fetched < t1) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int at = stage * kPieces + v * kOf;
        ring.fetch(at, x_at, col[v], f.hidden);
        if (GATES && has[v]) prefetch_gate(f, fetched, col[v]);
        if (normed()) ring.fetch(at + kA, dy_at, col[v], f.hidden);
        if (PRE && f.residual != nullptr) ring.fetch(at + 2 * kA, r_at, col[v], f.hidden);
        if (a.dsum != nullptr) ring.fetch(at + 2 * kA + kS, d_at, col[v], f.hidden);
      }
    }
    OwnRing::commit();
    ++fetched;
    x_at += f.x_stride;
    dy_at += a.dy_stride;
    r_at += f.residual_stride;
    d_at += a.dsum_stride;
  };
  {
    const float none[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < DEPTH * kPieces; i += 2) ring.put(i, none);
  }
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) fetch(i);
  const Pair zero = Pair::of(0.0f);
  Pair kept_w[4], kept_pre[4];
  const auto set_w = [&](int v, const float (&p)[8]) {
    if constexpr (kKeep)
      pairs_of(p, kept_w);
    else
      ring.put(kW + 2 * v, p);
  };
  const auto get_params = [&](int v, Pair (&w)[4], Pair (&pre)[4]) {
    if constexpr (kKeep) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = kept_w[i], pre[i] = kept_pre[i];
    } else {
      get_pairs<float>(ring, kW + 2 * v, w);
      get_pairs<float>(ring, kPre + 2 * v, pre);
    }
  };
  Pair dpre[NV][4], sum_g[NV][4], dpost[GATES ? NV : 1][4];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) dpre[v][i] = sum_g[v][i] = dpost[GATES ? v : 0][i] = zero;
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = 0.0f;
    set_w(v, p);
    if (has[v] && normed()) load_param<8>(f.pre, col[v], f.params_f32, p);
    if constexpr (kKeep)
      pairs_of(p, kept_pre);
    else
      ring.put(kPre + 2 * v, p);
  }
  // the tokens from which on another row of the gate holds
  int gate_row = 0, gate_end = t0;
  int stage = 0;
  float r1 = f.post && t0 < t1 ? f.post_rstd[t0] : 1.0f;
  float r2 = normed() && t0 < t1 ? f.pre_rstd[t0] : 0.0f;
  for (int t = t0; t < t1; ++t) {
    if (t >= gate_end) {
      gate_row = f.gate ? int(uint32_t(t) / uint32_t(f.gate_rows)) : 0;
      gate_end = f.gate ? int(min(int64_t(gate_row + 1) * f.gate_rows, int64_t(t1))) : t1;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (has[v]) {
          float p[8];
          load_factor(f, col[v], gate_row * f.gate_stride, p);
          set_w(v, p);
        }
    }
    OwnRing::wait<DEPTH - 1>();
    // (x and dy are kept as they lie in memory: a bf16 pair in one register, not two)
    Pack8<A> px[NV], py[NV];
    Pair sn[NV][4], d[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = stage * kPieces + v * kOf;
      ring.get(at, px[v]);
      if constexpr (PRE) {
        ring.get(at + kA, py[v]);
        get_pairs<S>(ring, at + 2 * kA, sn[v]);
      }
      get_pairs<S>(ring, at + 2 * kA + kS, d[v]);
    }
    fetch(stage);
    stage = stage + 1 == DEPTH ? 0 : stage + 1;
    const int next = t + 1 < t1 ? t + 1 : t;
    const float next_r1 = f.post ? f.post_rstd[next] : 1.0f;
    const float next_r2 = normed() ? f.pre_rstd[next] : 0.0f;
    Pair sa = zero, sb = zero, sc = zero;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      Pair w[4], pre[4], x[4], dy[4];
      pairs_of(px[v], x);
      if constexpr (PRE) pairs_of(py[v], dy);
      get_params(v, w, pre);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Pair z = w[i] * (x[i] * Pair::of(r1));
        if constexpr (!PRE) {
          sb = fma2(z, d[v][i], sb);
        } else {
          const Pair e = dy[i] * pre[i];
          sn[v][i] = (sn[v][i] + z) * Pair::of(r2);
          d[v][i] = fma2(Pair::of(r2), e, d[v][i]);
          sa = fma2(e, sn[v][i], sa);
          sb = fma2(z, d[v][i], sb);
          sc = fma2(z, sn[v][i], sc);
        }
      }
    }
    float k = 0.0f, m1;
    if constexpr (PRE) {
      float sum[3] = {sa.sum(), sb.sum(), sc.sum()};
      g.sums<3>(sum, buf, turn);
      k = r2 * (sum[0] * inv);
      m1 = (sum[1] - k * sum[2]) * inv;
    } else {
      float sum[1] = {sb.sum()};
      g.sums<1>(sum, buf, turn);
      m1 = sum[0] * inv;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      Pair w[4], pre[4], o[4], x[4], dy[4];
      pairs_of(px[v], x);
      if constexpr (PRE) pairs_of(py[v], dy);
      get_params(v, w, pre);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Pair xn = x[i] * Pair::of(r1);
        if constexpr (PRE) {
          d[v][i] = fma2(Pair::of(-k), sn[v][i], d[v][i]);
          dpre[v][i] = fma2(dy[i], sn[v][i], dpre[v][i]);
        }
        sum_g[v][i] = fma2(xn, d[v][i], sum_g[v][i]);
        o[i] = w[i] * d[v][i];
        if (f.post != nullptr) o[i] = Pair::of(r1) * fma2(Pair::of(-m1), xn, o[i]);
      }
      if (a.dresidual != nullptr)
        store8_warp(static_cast<S*>(a.dresidual) + (t * a.dresidual_stride + col[v]), has[v], d[v]);
      store8_warp(static_cast<A*>(a.dx) + (t * a.dx_stride + col[v]), has[v], o);
    }
    r1 = next_r1, r2 = next_r2;
    if (t + 1 < gate_end) continue;
    // the last token with this gate here
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!has[v]) continue;
      float p[8], q[8], s[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) sum_g[v][i].get(s[2 * i], s[2 * i + 1]), sum_g[v][i] = zero;
      if (f.gate != nullptr) {
        factor_of(f, f.post, col[v], p);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] *= s[i];
        store_gate<8>(a, n, t, worker, col[v], p);
      }
      if (f.post == nullptr) continue;
      factor_of(f, f.gate, gate_row * f.gate_stride + col[v], q);
      if constexpr (GATES) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dpost[v][i] = fma2(Pair::of(q[2 * i], q[2 * i + 1]), Pair::of(s[2 * i], s[2 * i + 1]),
                             dpost[v][i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] *= s[i];
        store_piece<8>(n.post_part + worker * f.hidden + col[v], q);
      }
    }
  }
  OwnRing::wait<0>();
  if (t0 >= t1) return;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (!has[v]) continue;
    if (normed()) store_pairs(n.pre_part + worker * f.hidden + col[v], dpre[v]);
    if (GATES && f.post != nullptr)
      store_pairs(n.post_part + worker * f.hidden + col[v], dpost[GATES ? v : 0]);
  }
}

// Rows of up to 4096 columns that need not lie on 16 bytes, as norm_few_kernel has
// them: eight columns per thread, E neighbouring ones of each 32 E of the row's
// threads; the next row is loaded while one is worked on.  (In two kernels, a column
// per thread: 838 us for 16384 x 4095 of bf16.)
template <typename A, typename S, int E, bool PRE>
__global__ void __launch_bounds__(512, 1) norm_backward_few_kernel(const NormBackArgs a,
                                                                   const BackShape n, int warps) {
  constexpr int U = 8 / E;
  __shared__ __align__(16) float buf[2 * 8 * 48];           // of up to eight rows
  for (int i = threadIdx.x; i < 2 * 8 * 48; i += blockDim.x) buf[i] = 0.0f;
  __syncthreads();
  int turn = 0;
  const NormArgs& f = a.f;
  const RowGroup g = RowGroup::of(warps);
  const int first = g.tid * E, stride = warps * 32 * E;
  const int64_t worker = int64_t(blockIdx.x) * (int(blockDim.x) / (warps * 32)) + g.index;
  const int t0 = int(min(worker * n.per_worker, int64_t(f.tokens)));
  const int t1 = min(t0 + n.per_worker, f.tokens);
  const float inv = 1.0f / float(f.hidden);
  Few<A, E> px[U], py[U];
  Few<S, E> pr[U], pd[U];
  const auto load = [&](int t) {
    const A* x = static_cast<const A*>(f.x) + (t * f.x_stride + first);
    const A* y = static_cast<const A*>(a.dy) + (t * a.dy_stride + first);
    const S* r = static_cast<const S*>(f.residual) + (t * f.residual_stride + first);
    const S* d = static_cast<const S*>(a.dsum) + (t * a.dsum_stride + first);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool has = t < t1 && first + i * stride < f.hidden;
      px[i].zero(), py[i].zero(), pr[i].zero(), pd[i].zero();
      if (has) px[i].load(x + i * stride);
      if (PRE && has) py[i].load(y + i * stride);
      if (PRE && has && f.residual != nullptr) pr[i].load(r + i * stride);
      if (has && a.dsum != nullptr) pd[i].load(d + i * stride);
    }
  };
  load(t0);
  float w[U][E], pre[U][E], dpre[U][E], dpost[U][E], sum_g[U][E];
#pragma unroll
  for (int i = 0; i < U; ++i) {
#pragma unroll
    for (int e = 0; e < E; ++e) w[i][e] = pre[i][e] = dpre[i][e] = dpost[i][e] = sum_g[i][e] = 0.0f;
    if (PRE && first + i * stride < f.hidden)
      load_few_param<E>(f.pre, first + i * stride, f.params_f32, pre[i]);
  }
  int gate_row = 0, gate_end = t0;
  for (int t = t0; t < t1; ++t) {
    if (t >= gate_end) {
      gate_row = f.gate ? int(uint32_t(t) / uint32_t(f.gate_rows)) : 0;
      gate_end = f.gate ? int(min(int64_t(gate_row + 1) * f.gate_rows, int64_t(t1))) : t1;
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (first + i * stride < f.hidden)
          load_few_factor<E>(f, first + i * stride, gate_row * f.gate_stride, w[i]);
    }
    float xn[U][E], sn[U][E], dy[U][E], d[U][E];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      px[i].get(xn[i]);
      py[i].get(dy[i]);
      pr[i].get(sn[i]);
      pd[i].get(d[i]);
    }
    load(t + 1);
    const float r1 = f.post ? f.post_rstd[t] : 1.0f, r2 = PRE ? f.pre_rstd[t] : 0.0f;
    float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        xn[i][e] *= r1;
        const float z = w[i][e] * xn[i][e];
        if constexpr (PRE) {
          const float q = dy[i][e] * pre[i][e];
          sn[i][e] = (sn[i][e] + z) * r2;
          d[i][e] = fmaf(r2, q, d[i][e]);
          sum[0] = fmaf(q, sn[i][e], sum[0]);
          sum[2] = fmaf(z, sn[i][e], sum[2]);
        }
        sum[1] = fmaf(z, d[i][e], sum[1]);
      }
    }
    float k = 0.0f, m1;
    if constexpr (PRE) {
      g.sums<3>(sum, buf, turn);
      k = r2 * (sum[0] * inv);
      m1 = (sum[1] - k * sum[2]) * inv;
    } else {
      float only[1] = {sum[1]};
      g.sums<1>(only, buf, turn);
      m1 = only[0] * inv;
    }
    S* dres = static_cast<S*>(a.dresidual) + (t * a.dresidual_stride + first);
    A* dx = static_cast<A*>(a.dx) + (t * a.dx_stride + first);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if constexpr (PRE) {
          d[i][e] = fmaf(-k, sn[i][e], d[i][e]);
          dpre[i][e] = fmaf(dy[i][e], sn[i][e], dpre[i][e]);
        }
        sum_g[i][e] = fmaf(xn[i][e], d[i][e], sum_g[i][e]);
        o[e] = w[i][e] * d[i][e];
        if (f.post != nullptr) o[e] = r1 * fmaf(-m1, xn[i][e], o[e]);
      }
      if (first + i * stride >= f.hidden) continue;
      if (a.dresidual != nullptr) Few<S, E>::store(dres + i * stride, d[i]);
      Few<A, E>::store(dx + i * stride, o);
    }
    if (t + 1 < gate_end) continue;
    // the last token with this gate here
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int col = first + i * stride;
      if (col >= f.hidden) continue;
      float p[E], q[E];
#pragma unroll
      for (int e = 0; e < E; ++e) p[e] = q[e] = 1.0f;
      if (f.post != nullptr) load_few_param<E>(f.post, col, f.params_f32, p);
      if (f.gate != nullptr)
        load_few_param<E>(f.gate, gate_row * f.gate_stride + col, f.params_f32, q);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float scaled = f.scale * sum_g[i][e];
        dpost[i][e] = fmaf(q[e], scaled, dpost[i][e]);
        sum_g[i][e] = 0.0f;
        if (f.gate != nullptr) {
          const float v[1] = {p[e] * scaled};
          store_gate<1>(a, n, t, worker, col + e, v);
        }
      }
    }
  }
  if (t0 >= t1) return;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (first + i * stride >= f.hidden) continue;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t at = worker * f.hidden + first + i * stride + e;
      if (PRE) n.pre_part[at] = dpre[i][e];
      if (f.post != nullptr) n.post_part[at] = dpost[i][e];
    }
  }
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
  cta_sums<3>(sum, buf, turn);
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
    if (f.gate && (t + 1 == t1 || (t + 1) % f.gate_rows == 0)) {
      store_gate<W>(a, n, t, worker, col, dgate);
#pragma unroll
      for (int i = 0; i < W; ++i) dgate[i] = 0.0f;
    }
  }
  store_parts<W>(a, n, worker, col, dpre, dpost);
}

// The parts' sums: a CTA takes 32 columns of one result, its warps every eighth part
// (or every 32nd, of many short rows' workers), and joins them in their order.
__global__ void __launch_bounds__(1024) norm_join_kernel(const NormBackArgs a, const BackShape n,
                                                         int columns) {
  __shared__ float buf[32][33];
  const NormArgs& f = a.f;
  int64_t which = blockIdx.x / unsigned(columns);
  const int col = int(blockIdx.x % unsigned(columns)) * 32 + (threadIdx.x & 31);
  const int warp = threadIdx.x >> 5, warps = int(blockDim.x) >> 5;
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
    constexpr int kAtOnce = 10;       // 152 workers: two waits
    for (int64_t w = lo + warp; w < hi; w += kAtOnce * warps) {
      float v[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        v[i] = w + i * warps < hi ? __ldcs(from + (w + i * warps) * f.hidden + col) : 0.0f;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) sum += v[i];
    }
  }
  buf[warp][threadIdx.x & 31] = sum;
  __syncthreads();
  if (warp != 0 || col >= f.hidden) return;
  for (int i = 1; i < warps; ++i) sum += buf[i][threadIdx.x];
  if (f.params_f32)
    static_cast<float*>(to)[at + col] = sum;
  else
    static_cast<uint16_t*>(to)[at + col] = narrow<uint16_t>(sum);
}

// Workers of at most as many as are asked for, where there are the tokens.
void share_out(BackShape* n, int64_t tokens, int64_t most) {
  n->per_worker = int32_t((tokens + most - 1) / most);
  n->workers = int32_t((tokens + n->per_worker - 1) / n->per_worker);
}

// Rows of one kernel: eight columns per thread up to 4096, and CTAs of 512 threads
// (with twice as many per thread the accumulators spill, and fewer rows are under way:
// 181 us).
RowShape whole_shape(int64_t hidden) { return row_shape(hidden, hidden <= 4096 ? 1 : 2, 16); }

// The most workers: a row of threads each, or the CTAs along the tokens.
int64_t whole_workers(int64_t hidden, int sms) { return int64_t(sms) * whole_shape(hidden).rows; }
int64_t column_workers(int64_t hidden, int width, int sms) {
  const int64_t pieces = (hidden + 256 * width - 1) / (256 * width);
  return (int64_t(sms) * 4 + pieces - 1) / pieces;
}

template <typename A, typename S, int NV, int DEPTH, bool GATES, bool PRE>
fo_status launch_kernel(const NormBackArgs& a, const BackShape& n, const RowShape& s, int row_bytes,
                      cudaStream_t st) {
  constexpr auto kernel = norm_backward_kernel<A, S, NV, DEPTH, GATES, PRE>;
  const fo_status q = allow_smem<kernel>();
  if (q != FO_OK) return q;
  const int smem = DEPTH * row_bytes + (NV == 1 ? 0 : s.threads * NV * 64);
  kernel<<<unsigned((n.workers + s.rows - 1) / s.rows), s.threads, smem, st>>>(a, n, s.warps);
  return FO_OK;
}
template <typename A, typename S, int NV, int DEPTH>
fo_status launch_ring(const NormBackArgs& a, const BackShape& n, const RowShape& s, int row_bytes,
                      cudaStream_t st) {
  const bool gates = a.f.gate != nullptr && a.f.gate_rows < a.f.tokens;
  if (a.f.pre != nullptr)
    return gates ? launch_kernel<A, S, NV, DEPTH, true, true>(a, n, s, row_bytes, st)
                 : launch_kernel<A, S, NV, DEPTH, false, true>(a, n, s, row_bytes, st);
  return gates ? launch_kernel<A, S, NV, DEPTH, true, false>(a, n, s, row_bytes, st)
               : launch_kernel<A, S, NV, DEPTH, false, false>(a, n, s, row_bytes, st);
}

template <typename A, typename S, int E>
void launch_few(const NormBackArgs& a, const BackShape& n, const RowShape& s, cudaStream_t st) {
  const unsigned grid = unsigned((n.workers + s.rows - 1) / s.rows);
  if (a.f.pre != nullptr)
    norm_backward_few_kernel<A, S, E, true><<<grid, s.threads, 0, st>>>(a, n, s.warps);
  else
    norm_backward_few_kernel<A, S, E, false><<<grid, s.threads, 0, st>>>(a, n, s.warps);
}

template <typename A, typename S>
fo_status launch(const NormBackArgs& a, BackShape* n, float* workspace, bool vec, bool two,
                 int sms, cudaStream_t st) {
  const NormArgs& f = a.f;
  const int64_t H = f.hidden;
  const RowShape s = whole_shape(H <= 8192 ? H : 0);
  const int row = s.threads * s.nv * 16 * int(sizeof(A) + sizeof(S));
  const int params = s.nv == 1 ? 0 : s.threads * s.nv * 64;
  const bool whole = vec && H <= 8192 && 2 * row + params <= kBlockSmem;
  const bool few = !vec && H <= 4096;
  if (whole || few) {
    share_out(n, f.tokens, whole_workers(H, sms));
  } else {
    share_out(n, f.tokens, column_workers(H, vec ? 8 : 1, sms));
    n->means = reinterpret_cast<float2*>(workspace);
    workspace += (2 * int64_t(f.tokens) + 3) / 4 * 4;
  }
  n->pre_part = workspace;
  n->post_part = n->pre_part + n->workers * H;
  n->gate_part = n->post_part + n->workers * H;
  if (whole) {
    // four rows under way where they fit, as those of bf16 do
    if (s.nv == 2) return launch_ring<A, S, 2, 2>(a, *n, s, row, st);
    if constexpr (sizeof(A) == 4) {
      if (4 * row > kBlockSmem) return launch_ring<A, S, 1, 2>(a, *n, s, row, st);
    }
    return launch_ring<A, S, 1, 4>(a, *n, s, row, st);
  }
  if (few) {
    if (two)
      launch_few<A, S, 2>(a, *n, s, st);
    else
      launch_few<A, S, 1>(a, *n, s, st);
    return FO_OK;
  }
  if (vec) {
    const int pieces = int((H + 2047) / 2048);
    norm_means_kernel<A, S, 8><<<unsigned(f.tokens), 512, 0, st>>>(a, *n);
    norm_columns_kernel<A, S, 8><<<unsigned(n->workers * pieces), 256, 0, st>>>(a, *n, pieces);
  } else {
    const int pieces = int((H + 255) / 256), w = int((H + 31) / 32);
    norm_means_kernel<A, S, 1><<<unsigned(f.tokens), (w < 16 ? w : 16) * 32, 0, st>>>(a, *n);
    norm_columns_kernel<A, S, 1><<<unsigned(n->workers * pieces), 256, 0, st>>>(a, *n, pieces);
  }
  return FO_OK;
}

}  // namespace

// Both means of every token, and the workers' parts.
int64_t block_norm_workspace_bytes(int64_t tokens, int64_t hidden, int64_t gates) {
  if (hidden == 0) return 16;
  int64_t workers = column_workers(hidden, 8, kMaxSms);
  if (hidden <= 8192 && workers < whole_workers(hidden, kMaxSms))
    workers = whole_workers(hidden, kMaxSms);
  if (workers > tokens) workers = tokens;
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
  const bool two = norm_rows_on_two(f, type, stream_type) &&
                   rows_on_two(a.dsum, a.dsum_stride, stream_type) &&
                   rows_on_two(a.dy, a.dy_stride, type) && rows_on_two(a.dx, a.dx_stride, type) &&
                   rows_on_two(a.dresidual, a.dresidual_stride, stream_type);
  int sms = 0;
  fo_status q = sm_count(&sms);
  if (q != FO_OK) return q;
  if (sms > kMaxSms) sms = kMaxSms;
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
      q = launch<float, float>(a, &n, a.workspace, vec, two, sms, st);
    else if (stream_type == FO_TYPE_F32)
      q = launch<uint16_t, float>(a, &n, a.workspace, vec, two, sms, st);
    else
      q = launch<uint16_t, uint16_t>(a, &n, a.workspace, vec, two, sms, st);
  }
  if (q != FO_OK) return q;
  if (cudaGetLastError() != cudaSuccess) return FO_ERR_CUDA;
  // (16384 x 64 in bf16, 2432 workers: 37 us with eight warps, 20 with 32)
  if (results > 0)
    norm_join_kernel<<<unsigned(results * columns), n.workers > 160 ? 1024 : 256, 0, st>>>(
        a, n, int(columns));
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace fo
