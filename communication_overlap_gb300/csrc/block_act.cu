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
// The code of x, by its low byte; x / step is below 128 in magnitude.
__device__ __forceinline__ int code_of(float x, float inverse, bool bad) {
  return bad ? 0 : max(-127, min(127, __float2int_rn(x * inverse)));
}

__device__ __forceinline__ float gated(float g, float u, int act) {
  if (act == FO_ACT_SILU) return g / (1.0f + expf(-g)) * u;
  if (act == FO_ACT_RELU) return (g > 0.0f ? g : 0.0f) * u;
  return g * u;
}

__device__ __forceinline__ void gated_backward(float dh, float g, float u, int act, float& dg,
                                               float& du) {
  if (act == FO_ACT_SILU) {
    const float e = expf(-g);
    const float s = 1.0f / (1.0f + e);
    dg = dh * u * (s * (1.0f + g * (1.0f - s)));
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

// A thread's row and first column: of eight columns where VEC, else of one.
struct Place {
  int64_t row;
  int col;
  bool live;
};
__device__ __forceinline__ Place place(const ActArgs& a, int width) {
  const int piece = int(blockIdx.x % unsigned(a.pieces));
  const int64_t r0 = int64_t(blockIdx.x / unsigned(a.pieces)) * a.per_cta;
  const int local = a.pieces > 1 ? 0 : int(threadIdx.x) / a.chunks;
  const int c = a.pieces > 1 ? piece * kThreads + int(threadIdx.x) : int(threadIdx.x) % a.chunks;
  Place p;
  p.row = r0 + local;
  p.col = c * width;
  p.live = local < a.per_cta && p.row < a.rows && p.col < a.padded;
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

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) act_kernel(const ActArgs a) {
  constexpr int W = VEC ? 8 : 1;
  const Place p = place(a, W);
  const bool in = p.live && p.col < a.inter;
  const T* src = static_cast<const T*>(a.u) + p.row * a.u_stride + p.col;
  float g[W], u[W];
#pragma unroll
  for (int i = 0; i < W; ++i) g[i] = u[i] = 0.0f;
  if (in) {
    if constexpr (VEC) {
      Pack8<T> pg, pu;
      pg.load_once(src);
      pu.load_once(src + a.inter);
      pg.get(g);
      pu.get(u);
    } else {
      g[0] = widen(__ldcs(src));
      u[0] = widen(__ldcs(src + a.inter));
    }
    float h[W];
#pragma unroll
    for (int i = 0; i < W; ++i) h[i] = gated(g[i], u[i], a.act);
    T* dst = static_cast<T*>(a.h) + p.row * a.h_stride + p.col;
    if constexpr (VEC)
      store8(dst, h);
    else
      *dst = narrow<T>(h[0]);
  }
  if (a.codes == nullptr) return;
  uint32_t mg = 0, mu = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    mg = max(mg, __float_as_uint(g[i]) & 0x7fffffffu);
    mu = max(mu, __float_as_uint(u[i]) & 0x7fffffffu);
  }
  const uint32_t sg = step_byte(block_max<VEC>(mg)), su = step_byte(block_max<VEC>(mu));
  if (!p.live) return;
  const float ig = inverse_step(sg), iu = inverse_step(su);
  int8_t* cg = a.codes + p.row * 2 * a.padded + p.col;
  if constexpr (VEC) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      q[i] = q[2 + i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        q[i] |= uint32_t(code_of(g[4 * i + j], ig, sg == 255u) & 255) << (8 * j);
        q[2 + i] |= uint32_t(code_of(u[4 * i + j], iu, su == 255u) & 255) << (8 * j);
      }
    }
    __stcs(reinterpret_cast<uint2*>(cg), make_uint2(q[0], q[1]));
    __stcs(reinterpret_cast<uint2*>(cg + a.padded), make_uint2(q[2], q[3]));
  } else {
    cg[0] = int8_t(code_of(g[0], ig, sg == 255u));
    cg[a.padded] = int8_t(code_of(u[0], iu, su == 255u));
  }
  if (p.col % kCheckpointBlock == 0) {
    const int blocks = a.padded / kCheckpointBlock;
    uint8_t* s = a.scales + p.row * 2 * blocks + p.col / kCheckpointBlock;
    s[0] = uint8_t(sg);
    s[blocks] = uint8_t(su);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) act_backward_kernel(const ActArgs a, const void* dh,
                                                               void* du) {
  constexpr int W = VEC ? 8 : 1;
  const Place p = place(a, W);
  if (!p.live || p.col >= a.inter) return;
  const T* src = static_cast<const T*>(dh) + p.row * a.h_stride + p.col;
  const int8_t* cg = a.codes + p.row * 2 * a.padded + p.col;
  const int blocks = a.padded / kCheckpointBlock;
  const uint8_t* s = a.scales + p.row * 2 * blocks + p.col / kCheckpointBlock;
  float d[W], g[W], u[W];
  uint2 qg, qu;
  if constexpr (VEC) {
    Pack8<T> v;
    v.load_once(src);
    qg = __ldcs(reinterpret_cast<const uint2*>(cg));
    qu = __ldcs(reinterpret_cast<const uint2*>(cg + a.padded));
    v.get(d);
  } else {
    d[0] = widen(__ldcs(src));
    qg.x = uint8_t(cg[0]), qu.x = uint8_t(cg[a.padded]);
  }
  const float vg = step_value(__ldg(s)), vu = step_value(__ldg(s + blocks));
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const uint32_t wg = i < 4 ? qg.x : qg.y, wu = i < 4 ? qu.x : qu.y;
    g[i] = float(int8_t(wg >> (8 * (i & 3)))) * vg;
    u[i] = float(int8_t(wu >> (8 * (i & 3)))) * vu;
  }
  float og[W], ou[W];
#pragma unroll
  for (int i = 0; i < W; ++i) gated_backward(d[i], g[i], u[i], a.act, og[i], ou[i]);
  T* dst = static_cast<T*>(du) + p.row * a.u_stride + p.col;
  if constexpr (VEC) {
    store8(dst, og);
    store8(dst + a.inter, ou);
  } else {
    dst[0] = narrow<T>(og[0]);
    dst[a.inter] = narrow<T>(ou[0]);
  }
}

bool on_16(const void* p, int64_t stride, fo_type type) {
  const int64_t size = type == FO_TYPE_BF16 ? 2 : 4;
  return ((reinterpret_cast<uintptr_t>(p) | uintptr_t(stride * size)) & 15) == 0;
}

// The grid over rows x padded columns, a chunk of `width` columns per thread;
// false where it has too many CTAs.
bool grid_of(ActArgs* a, int width, int64_t* grid) {
  const int64_t chunks = a->padded / width;
  a->pieces = int32_t((chunks + kThreads - 1) / kThreads);
  a->chunks = int32_t(chunks < kThreads ? chunks : kThreads);
  a->per_cta = a->pieces > 1 ? 1 : kThreads / a->chunks;
  *grid = (int64_t(a->rows) + a->per_cta - 1) / a->per_cta * a->pieces;
  return *grid < (int64_t(1) << 31);
}

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
  int64_t grid = 0;
  if (!grid_of(&a, vec ? 8 : 1, &grid)) return FO_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned n = unsigned(grid);
  if (type == FO_TYPE_BF16) {
    if (vec)
      act_kernel<uint16_t, true><<<n, kThreads, 0, st>>>(a);
    else
      act_kernel<uint16_t, false><<<n, kThreads, 0, st>>>(a);
  } else {
    if (vec)
      act_kernel<float, true><<<n, kThreads, 0, st>>>(a);
    else
      act_kernel<float, false><<<n, kThreads, 0, st>>>(a);
  }
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
  int64_t grid = 0;
  if (!grid_of(&a, vec ? 8 : 1, &grid)) return FO_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned n = unsigned(grid);
  if (type == FO_TYPE_BF16) {
    if (vec)
      act_backward_kernel<uint16_t, true><<<n, kThreads, 0, st>>>(a, dh, du);
    else
      act_backward_kernel<uint16_t, false><<<n, kThreads, 0, st>>>(a, dh, du);
  } else {
    if (vec)
      act_backward_kernel<float, true><<<n, kThreads, 0, st>>>(a, dh, du);
    else
      act_backward_kernel<float, false><<<n, kThreads, 0, st>>>(a, dh, du);
  }
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace fo
