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
// Both passes move each byte once and HBM bounds them: 32768 x 14336 of bf16, 3.79 GB
// each, 584 us forward (6.5 TB/s) and 540 back (7.0).  Two rows of 14336 take 1.6 us on
// the device.
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

// k / (1 + e^-kg), k = kScale of T: times g it is the silu of kg.  With fp32 outputs k = 1,
// by expf and a division.  With bf16 ones, which are rounded by 2^-9, by one power of two,
// and k = 2^8, so that the reciprocal has no number to flush while the power is one: without,
// silu was 0 from -87.3 on.  (The power's argument is rounded twice and itself off by
// 2^-22: with the reciprocal's 2^-23 off by less than (|kg| + 4) 2^-22.)  A third of
// expf's instructions, where those bind.
template <typename T>
constexpr float kScale = sizeof(T) == 2 ? 0x1p8f : 1.0f;
template <typename T>
constexpr float kPart = 1.0f / kScale<T>;
template <typename T>
__device__ __forceinline__ float scaled_sigmoid(float g) {
  if constexpr (sizeof(T) == 2) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * (-1.4426950408889634f * kScale<T>)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(fmaf(e, kPart<T>, kPart<T>)));
    return s;
  } else {
    return 1.0f / (1.0f + expf(-g));
  }
}

template <typename T>
__device__ __forceinline__ float gated(float g, float u, int act) {
  if (act == FO_ACT_SILU) {
    g *= kPart<T>;
    return g * scaled_sigmoid<T>(g) * u;
  }
  if (act == FO_ACT_RELU) return (g > 0.0f ? g : 0.0f) * u;
  return g * u;
}

template <typename T>
__device__ __forceinline__ void gated_backward(float dh, float g, float u, int act, float& dg,
                                               float& du) {
  if (act == FO_ACT_SILU) {
    g *= kPart<T>;
    const float s = scaled_sigmoid<T>(g);
    dg = dh * u * (s * fmaf(g, fmaf(s, -kPart<T>, 1.0f), kPart<T>));
    du = dh * (g * s);
  } else if (act == FO_ACT_RELU) {
    dg = g > 0.0f ? dh * u : 0.0f;
    du = dh * (g > 0.0f ? g : 0.0f);
  } else {
    dg = dh * u;
    du = dh * g;
  }
}

// The same for eight columns whose g and u are codes; of silu two values per
// instruction.
__device__ __forceinline__ Pair code_pair(uint32_t flipped, int i, float step) {
  const Pair v = Pair::of(__uint_as_float(__byte_perm(flipped, 0x4b000000u, 0x7440 + 2 * i)),
                          __uint_as_float(__byte_perm(flipped, 0x4b000000u, 0x7441 + 2 * i)));
  return (v + Pair::of(-8388736.0f)) * Pair::of(step);
}
template <typename T>
__device__ __forceinline__ void gated_backward(const Pack8<T>& dh, uint2 gate, uint2 up,
                                               float gate_step, float up_step, int act,
                                               float (&dg)[8], float (&du)[8]) {
  if (act == FO_ACT_SILU) {
    Pair d[4];
    pairs_of(dh, d);
    const uint32_t qg[2] = {gate.x ^ 0x80808080u, gate.y ^ 0x80808080u};
    const uint32_t qu[2] = {up.x ^ 0x80808080u, up.y ^ 0x80808080u};
    const float part_step = gate_step * kPart<T>;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Pair g = code_pair(qg[i / 2], i & 1, part_step), u = code_pair(qu[i / 2], i & 1, up_step);
      float a, b;
      g.get(a, b);
      const Pair s = Pair::of(scaled_sigmoid<T>(a), scaled_sigmoid<T>(b));
      const Pair slope = s * fma2(g, fma2(s, Pair::of(-kPart<T>), Pair::of(1.0f)), Pair::of(kPart<T>));
      (d[i] * u * slope).get(dg[2 * i], dg[2 * i + 1]);
      (d[i] * (g * s)).get(du[2 * i], du[2 * i + 1]);
    }
  } else {
    float d[8], g[8], u[8];
    dh.get(d);
    values_of(gate, gate_step, g);
    values_of(up, up_step, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) gated_backward<T>(d[i], g[i], u[i], act, dg[i], du[i]);
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

// A thread's first row and first of eight columns.  It has `rows` rows, `per_cta` apart.
struct Place {
  int64_t row;
  int col;
  bool live;      // the column exists, and the thread has a row's place
};
__device__ __forceinline__ Place place(const ActArgs& a, int rows) {
  const int piece = int(blockIdx.x % unsigned(a.pieces));
  const int64_t r0 = int64_t(blockIdx.x / unsigned(a.pieces)) * a.per_cta * rows;
  const int local = a.pieces > 1 ? 0 : int(threadIdx.x) / a.chunks;
  const int c = a.pieces > 1 ? piece * kThreads + int(threadIdx.x) : int(threadIdx.x) % a.chunks;
  Place p;
  p.row = r0 + local;
  p.col = c * 8;
  p.live = local < a.per_cta && p.col < a.padded;
  return p;
}

// The largest over the four neighbouring lanes that hold a block of 32.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
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
  const Place p = place(a, ROWS);
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
    const uint32_t mg = block_max(amax_of(pg[r])), mu = block_max(amax_of(pu[r]));
    if (!live) continue;
    const uint32_t sg = step_byte(mg), su = step_byte(mu);
    int8_t* to = a.codes + row * 2 * a.padded + p.col;
    __stcs(reinterpret_cast<uint2*>(to), codes_of(g, mg, sg));
    __stcs(reinterpret_cast<uint2*>(to + a.padded), codes_of(u, mu, su));
    store_scales(a, row, p.col, sg, su);
  }
}

// Rows that need not lie on 16 bytes: a warp takes kUnits times 32 E columns of a row, a
// lane E neighbouring ones of each 32 E, so that its loads and stores are of
// neighbouring addresses (one column per thread took 325 us for 16384 x 4095 of bf16).
constexpr int kUnits = 8;

// The largest over the lanes that hold a block of 32 columns.
template <int E>
__device__ __forceinline__ uint32_t few_max(uint32_t m) {
  if constexpr (E == 1) {
    return __reduce_max_sync(0xffffffffu, m);
  } else {
#pragma unroll
    for (int o = 1; o < 32 / E; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  }
}

// A warp's row and first column.
struct WarpPlace {
  int64_t row;
  int col;
};
template <int E>
__device__ __forceinline__ WarpPlace warp_place(const ActArgs& a) {
  const int64_t item = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  return {item / a.pieces, int(item % a.pieces) * kUnits * 32 * E};
}

template <typename T, int E>
__global__ void __launch_bounds__(kThreads) act_any_kernel(const ActArgs a) {
  const WarpPlace p = warp_place<E>(a);
  if (p.row >= a.rows) return;
  const int lane = threadIdx.x & 31, first = p.col + lane * E;
  const T* src = static_cast<const T*>(a.u) + p.row * a.u_stride + first;
  T* dst = static_cast<T*>(a.h) + p.row * a.h_stride + first;
  Few<T, E> pg[kUnits], pu[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    pg[i].zero();
    pu[i].zero();
    if (first + i * 32 * E < a.inter) {
      pg[i].load(src + i * 32 * E);
      pu[i].load(src + a.inter + i * 32 * E);
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int col = first + i * 32 * E;
    if (p.col + i * 32 * E >= a.padded) break;      // (the same for the warp)
    float g[E], u[E], h[E];
    pg[i].get(g);
    pu[i].get(u);
    if (col < a.inter) {
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] = gated<T>(g[e], u[e], a.act);
      Few<T, E>::store(dst + i * 32 * E, h);
    }
    if (a.codes == nullptr) continue;
    uint32_t mg = 0, mu = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      mg = max(mg, __float_as_uint(g[e]) & 0x7fffffffu);
      mu = max(mu, __float_as_uint(u[e]) & 0x7fffffffu);
    }
    const uint32_t sg = step_byte(few_max<E>(mg)), su = step_byte(few_max<E>(mu));
    if (col >= a.padded) continue;
    int8_t* to = a.codes + p.row * 2 * a.padded + col;
    const float ig = inverse_step(sg), iu = inverse_step(su);
    if constexpr (E == 1) {
      to[0] = int8_t(code_of(g[0], ig, sg));
      to[a.padded] = int8_t(code_of(u[0], iu, su));
    } else {
      const auto two = [](int x, int y) { return uint16_t((x & 255) | (y & 255) << 8); };
      *reinterpret_cast<uint16_t*>(to) = two(code_of(g[0], ig, sg), code_of(g[E - 1], ig, sg));
      *reinterpret_cast<uint16_t*>(to + a.padded) =
          two(code_of(u[0], iu, su), code_of(u[E - 1], iu, su));
    }
    store_scales(a, p.row, col, sg, su);
  }
}

// The same for the gradient, of one row per thread: with 32 registers eight CTAs of bf16
// are on an SM at once, and HBM is kept busy by warps in place of rows (32768 x 14336: two
// rows of 48 registers and one value per instruction took 625 us, one row of 47 620, of
// 40 582, this 540).
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 8 : 1)
    act_backward_kernel(const ActArgs a, const void* dh, void* du) {
  const Place p = place(a, 1);
  const int row = int(p.row);       // (of one per thread: below 2^31)
  const bool in = p.live && p.col < a.inter && row < a.rows;
  const int blocks = a.padded / kCheckpointBlock;
  Pack8<T> d;
  uint2 qg = make_uint2(0, 0), qu = make_uint2(0, 0);
  uint32_t sg = 0, su = 0;
  d.zero();
  if (in) {
    const int8_t* from = a.codes + int64_t(row) * 2 * a.padded + p.col;
    const uint8_t* s = a.scales + int64_t(row) * 2 * blocks + p.col / kCheckpointBlock;
    d.load_once(static_cast<const T*>(dh) + row * a.h_stride + p.col);
    qg = __ldcs(reinterpret_cast<const uint2*>(from));
    qu = __ldcs(reinterpret_cast<const uint2*>(from + a.padded));
    sg = __ldg(s);
    su = __ldg(s + blocks);
  }
  float og[8], ou[8];
  gated_backward(d, qg, qu, step_value(sg), step_value(su), a.act, og, ou);
  T* dst = static_cast<T*>(du) + row * a.u_stride + p.col;
  store8_warp(dst, in, og);
  store8_warp(dst + a.inter, in, ou);
}

template <typename T, int E>
__global__ void __launch_bounds__(kThreads) act_backward_any_kernel(const ActArgs a,
                                                                   const void* dh, void* du) {
  const WarpPlace p = warp_place<E>(a);
  if (p.row >= a.rows) return;
  const int lane = threadIdx.x & 31, first = p.col + lane * E;
  const int blocks = a.padded / kCheckpointBlock;
  const T* src = static_cast<const T*>(dh) + p.row * a.h_stride + first;
  T* dst = static_cast<T*>(du) + p.row * a.u_stride + first;
  const int8_t* codes = a.codes + p.row * 2 * a.padded + first;
  const uint8_t* scales = a.scales + p.row * 2 * blocks;
  Few<T, E> pd[kUnits];
  uint32_t qg[kUnits], qu[kUnits], sg[kUnits], su[kUnits];
  const auto load = [](const int8_t* p) {
    return E == 1 ? uint32_t(uint8_t(*p)) : uint32_t(*reinterpret_cast<const uint16_t*>(p));
  };
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int col = first + i * 32 * E;
    if (col >= a.inter) continue;
    pd[i].load(src + i * 32 * E);
    qg[i] = load(codes + i * 32 * E);
    qu[i] = load(codes + a.padded + i * 32 * E);
    sg[i] = __ldg(scales + col / kCheckpointBlock);
    su[i] = __ldg(scales + blocks + col / kCheckpointBlock);
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (first + i * 32 * E >= a.inter) continue;
    float d[E], og[E], ou[E];
    pd[i].get(d);
    const float vg = step_value(sg[i]), vu = step_value(su[i]);
#pragma unroll
    for (int e = 0; e < E; ++e)
      gated_backward<T>(d[e], float(int8_t(qg[i] >> (8 * e))) * vg,
                        float(int8_t(qu[i] >> (8 * e))) * vu, a.act, og[e], ou[e]);
    Few<T, E>::store(dst + i * 32 * E, og);
    Few<T, E>::store(dst + a.inter + i * 32 * E, ou);
  }
}

// The grid over rows x padded columns, a chunk of eight columns of `rows` rows per
// thread; false where it has too many CTAs.
bool grid_of(ActArgs* a, int rows, int64_t* grid) {
  const int64_t chunks = a->padded / 8;
  a->pieces = int32_t((chunks + kThreads - 1) / kThreads);
  a->chunks = int32_t(chunks < kThreads ? chunks : kThreads);
  a->per_cta = a->pieces > 1 ? 1 : kThreads / a->chunks;
  const int64_t of_cta = int64_t(a->per_cta) * rows;
  *grid = (int64_t(a->rows) + of_cta - 1) / of_cta * a->pieces;
  return *grid < (int64_t(1) << 31);
}

// The grid of warps over rows and pieces of kUnits * 32 * E columns.
bool grid_of_warps(ActArgs* a, int e, int64_t* grid) {
  const int width = kUnits * 32 * e;
  a->pieces = (a->padded + width - 1) / width;
  *grid = (int64_t(a->rows) * a->pieces + kThreads / 32 - 1) / (kThreads / 32);
  return *grid < (int64_t(1) << 31);
}

// Rows of a thread of act_kernel: two of bf16.
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
  const bool vec = inter % 8 == 0 && rows_on(u, u_stride, type, 16) &&
                   rows_on(h, h_stride, type, 16);
  const bool two = inter % 2 == 0 && rows_on_two(u, u_stride, type) &&
                   rows_on_two(h, h_stride, type);
  const bool bf16 = type == FO_TYPE_BF16;
  int64_t grid = 0;
  if (!(vec ? grid_of(&a, bf16 ? kRowsOf2 : kRowsOf4, &grid)
            : grid_of_warps(&a, two ? 2 : 1, &grid)))
    return FO_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned n = unsigned(grid);
  if (vec && bf16)
    act_kernel<uint16_t, kRowsOf2><<<n, kThreads, 0, st>>>(a);
  else if (vec)
    act_kernel<float, kRowsOf4><<<n, kThreads, 0, st>>>(a);
  else if (bf16 && two)
    act_any_kernel<uint16_t, 2><<<n, kThreads, 0, st>>>(a);
  else if (bf16)
    act_any_kernel<uint16_t, 1><<<n, kThreads, 0, st>>>(a);
  else if (two)
    act_any_kernel<float, 2><<<n, kThreads, 0, st>>>(a);
  else
    act_any_kernel<float, 1><<<n, kThreads, 0, st>>>(a);
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
  const bool vec = inter % 8 == 0 && rows_on(dh, dh_stride, type, 16) &&
                   rows_on(du, du_stride, type, 16);
  const bool two = inter % 2 == 0 && rows_on_two(dh, dh_stride, type) &&
                   rows_on_two(du, du_stride, type);
  const bool bf16 = type == FO_TYPE_BF16;
  int64_t grid = 0;
  if (!(vec ? grid_of(&a, 1, &grid)
            : grid_of_warps(&a, two ? 2 : 1, &grid)))
    return FO_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned n = unsigned(grid);
  if (vec && bf16)
    act_backward_kernel<uint16_t><<<n, kThreads, 0, st>>>(a, dh, du);
  else if (vec)
    act_backward_kernel<float><<<n, kThreads, 0, st>>>(a, dh, du);
  else if (bf16 && two)
    act_backward_any_kernel<uint16_t, 2><<<n, kThreads, 0, st>>>(a, dh, du);
  else if (bf16)
    act_backward_any_kernel<uint16_t, 1><<<n, kThreads, 0, st>>>(a, dh, du);
  else if (two)
    act_backward_any_kernel<float, 2><<<n, kThreads, 0, st>>>(a, dh, du);
  else
    act_backward_any_kernel<float, 1><<<n, kThreads, 0, st>>>(a, dh, du);
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace fo
