// The gated activation between an expert's projections, and its checkpoint of
// 8 bits per value.
//
//   h = act(g) u                          for a row [g | u] of 2 inter values
//   dg = dh u act'(g),  du = dh act(g)    g and u from the checkpoint
//   silu(g) = g / (1 + e^-g),  silu'(g) = s (1 + g (1 - s)),  s = 1 / (1 + e^-g)
//
// The checkpoint: per 32 values x_i of g or u, with a = max |x_i|, a step of
// 2^(floor(log2 a) - 6) and codes = the integer nearest x_i / step, at most 127
// in magnitude.  floor(log2 a) is a's exponent field and the step a power of
// two, so the only rounding is the one to an integer: at most half a step, a/128
// (one step, a/64, for magnitudes above 127.5 steps).  An e4m3 form of the same
// size has 4 significant bits per value: three times the error on normal data.
//
// Both passes move each byte once and HBM bounds them.
#include <cuda_runtime.h>

#include "block_common.cuh"

namespace fo {

namespace {

constexpr int kThreads = 256;

// The step's exponent byte from the largest magnitude's bits (a step is
// 2^(byte - 127); 255: the block holds an infinity or a NaN).
__device__ __forceinline__ uint32_t step_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  if (e == 255u) return 255u;
  return e > 6u ? e - 6u : 0u;
}
__device__ __forceinline__ float inverse_step(uint32_t s) {
  return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
}
__device__ __forceinline__ float step_value(uint32_t s) {
  if (s == 255u) return __uint_as_float(0x7fffffffu);
  return s == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23);
}
// Whether some code of the block is not simply the nearest integer: its largest
// magnitude is 127.5 steps or more, or no number.
__device__ __forceinline__ bool rare_block(uint32_t amax_bits) {
  return (amax_bits & 0x7fffffu) >= 0x7f0000u || amax_bits >= 0x7f800000u;
}
__device__ __forceinline__ int code_of(float x, float inverse, uint32_t step) {
  return step == 255u ? 0 : max(-127, min(127, __float2int_rn(x * inverse)));
}

// Eight codes, the first in the lowest byte.  x / step + 1.5 2^23 has the nearest
// integer, ties to even, in its lowest bits: one instruction per code where a
// conversion to an integer has a fourth of its rate.
__device__ __forceinline__ uint2 codes_of(const float (&x)[8], uint32_t amax_bits, uint32_t step) {
  const float inverse = inverse_step(step);
  uint32_t w[8];
  if (!rare_block(amax_bits)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(fmaf(x[i], inverse, 12582912.0f));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = uint32_t(code_of(x[i], inverse, step));
  }
  const auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
  };
  return make_uint2(four(w[0], w[1], w[2], w[3]), four(w[4], w[5], w[6], w[7]));
}
// The values of eight codes: a byte + 128 as the low bits of 2^23 is one permutation.
__device__ __forceinline__ void values_of(uint2 codes, float step, float (&v)[8]) {
  const uint32_t q[2] = {codes.x ^ 0x80808080u, codes.y ^ 0x80808080u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = (__uint_as_float(__byte_perm(q[i / 4], 0x4b000000u, 0x7440 + (i & 3))) - 8388736.0f) *
           step;
}

// The largest magnitude's fp32 bits.
__device__ __forceinline__ uint32_t amax_of(const Pack8<uint16_t>& p) {
  uint32_t m = p.w[0].x & 0x7fff7fffu;
  asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(p.w[0].y & 0x7fff7fffu));
  asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(p.w[0].z & 0x7fff7fffu));
  asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(p.w[0].w & 0x7fff7fffu));
  return max(m << 16, m & 0xffff0000u);
}
__device__ __forceinline__ uint32_t amax_of(const Pack8<float>& p) {
  const uint32_t w[8] = {p.w[0].x, p.w[0].y, p.w[0].z, p.w[0].w,
                         p.w[1].x, p.w[1].y, p.w[1].z, p.w[1].w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
  return m;
}

// 1 / (1 + e^-g).  With fp32 outputs by expf and a division.  With bf16 ones, which are rounded by
// 2^-9, by one power of two (its argument is rounded twice and itself off by 2^-22: with
// the reciprocal's 2^-23 off by less than (|g| + 4) 2^-22): a third of the
// instructions, where those bind.
template <typename T>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (sizeof(T) == 2) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return s;
  } else {
    return 1.0f / (1.0f + expf(-g));
  }
}

template <typename T>
__device__ __forceinline__ float gated(float g, float u, int act) {
  if (act == FO_ACT_SILU) return g * sigmoid<T>(g) * u;
  if (act == FO_ACT_RELU) return (g > 0.0f ? g : 0.0f) * u;
  return g * u;
}

template <typename T>
__device__ __forceinline__ void gated_backward(float dh, float g, float u, int act, float& dg,
                                               float& du) {
  if (act == FO_ACT_SILU) {
    const float s = sigmoid<T>(g);
    dg = dh * u * (s * fmaf(g, 1.0f - s, 1.0f));
    du = dh * (g * s);
  } else if (act == FO_ACT_RELU) {
    dg = g > 0.0f ? dh * u : 0.0f;
    du = dh * (g > 0.0f ? g : 0.0f);
  } else {
    dg = dh * u;
    du = dh * g;
  }
}

struct ActArgs {
  const void* u;
  void* h;
  int64_t u_stride, h_stride;
  int8_t* codes;            // [rows][2][padded], NULL: no checkpoint
  uint8_t* scales;          // [rows][2][padded / 32]
  int32_t rows, inter, padded;
  int32_t act;
  int32_t pieces, chunks, per_cta;    // the grid's shape, in threads' chunks
};

// A thread's first row and first column: of eight columns where VEC, else of one.
// It has `rows` rows, `per_cta` apart.
struct Place {
  int64_t row;
  int col;
  bool live;      // the column exists, and the thread has a row's place
};
__device__ __forceinline__ Place place(const ActArgs& a, int width, int rows) {
  const int piece = int(blockIdx.x % unsigned(a.pieces));
  const int64_t r0 = int64_t(blockIdx.x / unsigned(a.pieces)) * a.per_cta * rows;
  const int local = a.pieces > 1 ? 0 : int(threadIdx.x) / a.chunks;
  const int c = a.pieces > 1 ? piece * kThreads + int(threadIdx.x) : int(threadIdx.x) % a.chunks;
  Place p;
  p.row = r0 + local;
  p.col = c * width;
  p.live = local < a.per_cta && p.col < a.padded;
  return p;
}

// Four neighbouring lanes (VEC) or a warp hold a block of 32.
template <bool VEC>
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  if constexpr (VEC) {
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  } else {
    return __reduce_max_sync(0xffffffffu, m);
  }
}

__device__ __forceinline__ void store_scales(const ActArgs& a, int64_t row, int col, uint32_t sg,
                                             uint32_t su) {
  if (col % kCheckpointBlock) return;
  const int blocks = a.padded / kCheckpointBlock;
  uint8_t* s = a.scales + row * 2 * blocks + col / kCheckpointBlock;
  s[0] = uint8_t(sg);
  s[blocks] = uint8_t(su);
}

// Rows of which everything lies on 16 bytes: eight columns per thread, of ROWS rows
// whose loads are all under way at once.
template <typename T, int ROWS>
__global__ void __launch_bounds__(kThreads) act_kernel(const ActArgs a) {
  const Place p = place(a, 8, ROWS);
  const bool in = p.live && p.col < a.inter;
  Pack8<T> pg[ROWS], pu[ROWS];
  const T* src = static_cast<const T*>(a.u) + p.row * a.u_stride + p.col;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (in && p.row + r * a.per_cta < a.rows) {
      pg[r].load_once(src);
      pu[r].load_once(src + a.inter);
    } else {
      pg[r].zero();
      pu[r].zero();
    }
    src += a.per_cta * a.u_stride;
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int64_t row = p.row + r * a.per_cta;
    const bool live = p.live && row < a.rows;
    float g[8], u[8], h[8];
    pg[r].get(g);
    pu[r].get(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = gated<T>(g[i], u[i], a.act);
    store8_warp(static_cast<T*>(a.h) + row * a.h_stride + p.col, live && in, h);
    if (a.codes == nullptr) continue;
    const uint32_t mg = block_max<true>(amax_of(pg[r])), mu = block_max<true>(amax_of(pu[r]));
    if (!live) continue;
    const uint32_t sg = step_byte(mg), su = step_byte(mu);
    int8_t* to = a.codes + row * 2 * a.padded + p.col;
    __stcs(reinterpret_cast<uint2*>(to), codes_of(g, mg, sg));
    __stcs(reinterpret_cast<uint2*>(to + a.padded), codes_of(u, mu, su));
    store_scales(a, row, p.col, sg, su);
  }
}

// Any rows: a column per thread, a warp to a block of 32.
template <typename T>
__global__ void __launch_bounds__(kThreads) act_any_kernel(const ActArgs a) {
  const Place p = place(a, 1, 1);
  const bool live = p.live && p.row < a.rows, in = live && p.col < a.inter;
  const T* src = static_cast<const T*>(a.u) + p.row * a.u_stride + p.col;
  float g = 0.0f, u = 0.0f;
  if (in) {
    g = widen(__ldcs(src));
    u = widen(__ldcs(src + a.inter));
    static_cast<T*>(a.h)[p.row * a.h_stride + p.col] = narrow<T>(gated<T>(g, u, a.act));
  }
  if (a.codes == nullptr) return;
  const uint32_t mg = block_max<false>(__float_as_uint(g) & 0x7fffffffu);
  const uint32_t mu = block_max<false>(__float_as_uint(u) & 0x7fffffffu);
  if (!live) return;
  const uint32_t sg = step_byte(mg), su = step_byte(mu);
  int8_t* to = a.codes + p.row * 2 * a.padded + p.col;
  to[0] = int8_t(code_of(g, inverse_step(sg), sg));
  to[a.padded] = int8_t(code_of(u, inverse_step(su), su));
  store_scales(a, p.row, p.col, sg, su);
}

template <typename T, int ROWS>
__global__ void __launch_bounds__(kThreads) act_backward_kernel(const ActArgs a, const void* dh,
                                                               void* du) {
  const Place p = place(a, 8, ROWS);
  const bool in = p.live && p.col < a.inter;
  const int blocks = a.padded / kCheckpointBlock;
  Pack8<T> pd[ROWS];
  uint2 qg[ROWS], qu[ROWS];
  uint32_t sg[ROWS], su[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int64_t row = p.row + r * a.per_cta;
    if (!in || row >= a.rows) {
      pd[r].zero();
      qg[r] = qu[r] = make_uint2(0, 0);
      sg[r] = su[r] = 0;
      continue;
    }
    const int8_t* from = a.codes + row * 2 * a.padded + p.col;
    const uint8_t* s = a.scales + row * 2 * blocks + p.col / kCheckpointBlock;
    pd[r].load_once(static_cast<const T*>(dh) + row * a.h_stride + p.col);
    qg[r] = __ldcs(reinterpret_cast<const uint2*>(from));
    qu[r] = __ldcs(reinterpret_cast<const uint2*>(from + a.padded));
    sg[r] = __ldg(s);
    su[r] = __ldg(s + blocks);
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int64_t row = p.row + r * a.per_cta;
    float d[8], g[8], u[8], og[8], ou[8];
    pd[r].get(d);
    values_of(qg[r], step_value(sg[r]), g);
    values_of(qu[r], step_value(su[r]), u);
#pragma unroll
    for (int i = 0; i < 8; ++i) gated_backward<T>(d[i], g[i], u[i], a.act, og[i], ou[i]);
    T* dst = static_cast<T*>(du) + row * a.u_stride + p.col;
    store8_warp(dst, in && row < a.rows, og);
    store8_warp(dst + a.inter, in && row < a.rows, ou);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) act_backward_any_kernel(const ActArgs a,
                                                                   const void* dh, void* du) {
  const Place p = place(a, 1, 1);
  if (!p.live || p.row >= a.rows || p.col >= a.inter) return;
  const int blocks = a.padded / kCheckpointBlock;
  const int8_t* from = a.codes + p.row * 2 * a.padded + p.col;
  const uint8_t* s = a.scales + p.row * 2 * blocks + p.col / kCheckpointBlock;
  const float d = widen(__ldcs(static_cast<const T*>(dh) + p.row * a.h_stride + p.col));
  const float g = float(from[0]) * step_value(__ldg(s));
  const float u = float(from[a.padded]) * step_value(__ldg(s + blocks));
  float og, ou;
  gated_backward<T>(d, g, u, a.act, og, ou);
  T* dst = static_cast<T*>(du) + p.row * a.u_stride + p.col;
  dst[0] = narrow<T>(og);
  dst[a.inter] = narrow<T>(ou);
}

bool on_16(const void* p, int64_t stride, fo_type type) {
  const int64_t size = type == FO_TYPE_BF16 ? 2 : 4;
  return ((reinterpret_cast<uintptr_t>(p) | uintptr_t(stride * size)) & 15) == 0;
}

// The grid over rows x padded columns, a chunk of `width` columns of `rows` rows per
// thread; false where it has too many CTAs.
bool grid_of(ActArgs* a, int width, int rows, int64_t* grid) {
  const int64_t chunks = a->padded / width;
  a->pieces = int32_t((chunks + kThreads - 1) / kThreads);
  a->chunks = int32_t(chunks < kThreads ? chunks : kThreads);
  a->per_cta = a->pieces > 1 ? 1 : kThreads / a->chunks;
  const int64_t of_cta = int64_t(a->per_cta) * rows;
  *grid = (int64_t(a->rows) + of_cta - 1) / of_cta * a->pieces;
  return *grid < (int64_t(1) << 31);
}

// Rows of a thread: two of bf16.
constexpr int kRowsOf2 = 2, kRowsOf4 = 1;

int32_t padded_of(int64_t inter) {
  return int32_t((inter + kCheckpointBlock - 1) / kCheckpointBlock * kCheckpointBlock);
}

}  // namespace

fo_status launch_gated_act(const void* u, fo_type type, int64_t rows, int64_t inter,
                           int64_t u_stride, fo_activation act, void* h, int64_t h_stride,
                           void* codes, void* scales, void* stream) {
  ActArgs a{};
  a.u = u, a.h = h, a.u_stride = u_stride, a.h_stride = h_stride;
  a.codes = static_cast<int8_t*>(codes), a.scales = static_cast<uint8_t*>(scales);
  a.rows = int32_t(rows), a.inter = int32_t(inter), a.padded = padded_of(inter), a.act = act;
  const bool vec = inter % 8 == 0 && on_16(u, u_stride, type) && on_16(h, h_stride, type);
  const bool bf16 = type == FO_TYPE_BF16;
  int64_t grid = 0;
  if (!grid_of(&a, vec ? 8 : 1, !vec ? 1 : bf16 ? kRowsOf2 : kRowsOf4, &grid))
    return FO_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned n = unsigned(grid);
  if (vec && bf16)
    act_kernel<uint16_t, kRowsOf2><<<n, kThreads, 0, st>>>(a);
  else if (vec)
    act_kernel<float, kRowsOf4><<<n, kThreads, 0, st>>>(a);
  else if (bf16)
    act_any_kernel<uint16_t><<<n, kThreads, 0, st>>>(a);
  else
    act_any_kernel<float><<<n, kThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

fo_status launch_gated_act_backward(const void* dh, fo_type type, int64_t rows, int64_t inter,
                                    int64_t dh_stride, fo_activation act, const void* codes,
                                    const void* scales, void* du, int64_t du_stride,
                                    void* stream) {
  ActArgs a{};
  a.u_stride = du_stride, a.h_stride = dh_stride;
  a.codes = static_cast<int8_t*>(const_cast<void*>(codes));
  a.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
  a.rows = int32_t(rows), a.inter = int32_t(inter), a.padded = padded_of(inter), a.act = act;
  const bool vec = inter % 8 == 0 && on_16(dh, dh_stride, type) && on_16(du, du_stride, type);
  const bool bf16 = type == FO_TYPE_BF16;
  int64_t grid = 0;
  if (!grid_of(&a, vec ? 8 : 1, !vec ? 1 : bf16 ? kRowsOf2 : kRowsOf4, &grid))
    return FO_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned n = unsigned(grid);
  if (vec && bf16)
    act_backward_kernel<uint16_t, kRowsOf2><<<n, kThreads, 0, st>>>(a, dh, du);
  else if (vec)
    act_backward_kernel<float, kRowsOf4><<<n, kThreads, 0, st>>>(a, dh, du);
  else if (bf16)
    act_backward_any_kernel<uint16_t><<<n, kThreads, 0, st>>>(a, dh, du);
  else
    act_backward_any_kernel<float><<<n, kThreads, 0, st>>>(a, dh, du);
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace fo
