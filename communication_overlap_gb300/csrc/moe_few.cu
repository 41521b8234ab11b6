// A whole expert layer for a few tokens, in one kernel:
//   ids, w = top-k softmax of x . router^T,
//   h = act(G_e x) * (U_e x),  y[t] = sum_s w_s D_e h.
//
// A generation step reads every weight of every expert that a token reaches
// and does almost nothing with it: HBM bounds it, and what must not happen is
// that the reads pause.  So:
//  * One persistent CTA per SM (a cooperative launch).  Four warps copy
//    weights through a deep ring of stages (128 rows x 128 columns of bf16, or x
//    256 of 4 bits), eight warps consume them with mma.sync, a few tokens being
//    the narrow side (16 weight rows x 8 tokens x 16 columns).
//  * Work is cut evenly, whatever the routing: the hidden rows of all reached
//    experts are one line of granules and CTA c takes the c-th part of it; the
//    output product is one line of (128 output rows, expert, stage of columns),
//    cut the same way.
//  * A warp's 16 rows are 8 gate rows and their 8 up rows, which puts both
//    sums of a hidden row in one thread: the activation happens in registers
//    and only the hidden values (a few rows) travel through memory, inside L2.
//  * Between the two products stands a grid barrier.  The ring fills with the
//    second product's weights before it; only the loads of h wait.
//  * Output rows shared by several CTAs are joined by the last of them to
//    finish, which adds the parts in CTA order: the same bits in every run.
//
// bf16 weights: copied 16 bytes per thread (cp.async: rows of any multiple of
// 16 bytes); bf16 products, h rounded to bf16 as an operand of such (x has no
// more bits).  4-bit weights: bulk copies of codes and scales as they are kept;
// codes become f16 in registers (exact), x and h are f16 (11 bits) with a
// power-of-two scale per token and per 32 values; a block's sum of 32 products
// starts at zero and is added times the scales in fp32.
//
// Measured (8 experts, hidden 4096, inter 14336, top 2; bytes are those of the
// reached experts' weights):
//   bf16   1 token 117 us (6.0 TB/s), 8 tokens 366 (6.7), 48 tokens 419 (6.7):
//          the reads, and 20 us around them (launch, router and choice 6, the two
//          barriers, the join)
//   4-bit  1 token 56 us (3.4 TB/s), 8 tokens 148 (4.5), 48 tokens 287 (2.6) while no
//          expert has more than 16, 350 with one of 17, 576 with one of all 48: the
//          cut is even in weights, and an expert's stages take longer by its tiles of
//          8 tokens.  No unit is near its limit (1 token: issue slots 28% busy, tensor
//          cores 10%).  With the products taken out 1 token still takes 47 us: copies,
//          barriers and the ends of tiles (2000 to 3000 cycles each), 16 us of it
//          outside the two products.  A stage's products, 800 to 900 cycles per 20 KB
//          (HBM 750 to 880) for one tile of tokens and nearly twice that for two, are
//          a chain of shared memory, decoding, two MMAs and scaling in 8 warps that
//          start together; they count with more tokens.  Tried: 16 warps that halve a
//          stage's columns or take turns at stages (no faster), operands taken half a
//          stage ahead (15% slower).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "moe_common.cuh"
#include "mx_common.cuh"
#include "tensor_core.cuh"
#include "tensor_map.h"

namespace fo {

namespace {

constexpr int kMaxCtas = 160;
constexpr int kMaxRowBlocks = 4096;     // blocks of 128 output rows
constexpr int kMaxStages = 16;
constexpr int kSmemLimit = 232448;
constexpr int kCopyWarps = 4;
constexpr int kYPitch = 132;            // floats per token of the outputs' sums
// Columns of the weights per stage: 256 bytes of a bf16 row, 128 of a 4-bit one.
template <bool MX>
constexpr int kStageK = MX ? 256 : 128;
// A token's share of a 4-bit stage, in memory and in shared memory: 256 f16
// values, their eight scales (fp32), and what shifts the next token by 16 banks.
constexpr int kMxToken = 576;
constexpr int kMxScales = 16384, kMxTokens = kMxScales + 4096;   // offsets in a stage

template <int N>
struct Const {
  static constexpr int value = N;
};

// n items cut into g even parts: first(c) = n * c / g.  (Every item is 128 bytes
// of weights or more, so their number fits 32 bits; a 64-bit division is 400
// cycles.)
struct Cut {
  int32_t n, g, base, rem;
  uint32_t inverse;   // ceil(2^24 / g): x / g = x * inverse >> 24 for x < g * g, g <= 160
  __device__ __forceinline__ Cut(int n_, int g_, uint32_t inverse_)
      : n(n_), g(g_), base(n_ / g_), rem(n_ - base * g_), inverse(inverse_) {}
  __device__ __forceinline__ int first(int c) const {
    return base * c + int(uint32_t(rem * c) * inverse >> 24);
  }
  // the part that item x lies in
  __device__ __forceinline__ int owner(int x) const {
    int c = min(int(float(x) * float(g) / float(n)), g - 1);
    while (first(c + 1) <= x) ++c;
    while (first(c) > x) --c;
    return c;
  }
};

struct FewArgs {
  CUtensorMap map_w1[2], map_w2;   // 4-bit: boxes of 128 bytes x 32, 64 and 64 rows
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* router;
  const uint8_t *w1, *w2;  // weights: bf16 or codes
  const uint8_t *s1, *s2;  // 4-bit: scales
  uint16_t* y;
  int64_t y_stride;
  int32_t T, H, I, E, K, renormalize, act;
  int32_t w1_rows, w2_rows;   // rows of an expert's matrices as stored
  int32_t ring_bytes;
  uint32_t inverse_g;
  int32_t off_lists, off_y, off_bar;      // shared memory offsets
  uint32_t* barrier;          // [0], [1] counts, [2] leave
  int32_t* done;              // [row blocks] parts finished
  float* logits;              // [T][E]
  uint16_t* h;                // bf16: [rows][I]
  uint8_t *xq, *hq;           // 4-bit: [stage of columns][token or row] of kMxToken bytes
  float* x_scale;             // 4-bit: [T]
  int32_t h_rows;             // rows of hq per stage
  int32_t hp, ip;             // 4-bit: columns of xq and hq, whole stages
  int32_t hb, ib;             // and blocks of 128 columns of the weights
  float* parts;               // [kMaxCtas + row blocks][T][128]
  int32_t* status;
};

// The routing as every CTA keeps it in shared memory.
struct Lists {
  float* weight;      // [P] weight of row r (rows sorted by expert, token, slot)
  float* pair_weight; // [P]
  float* x_scale;     // [T] 4-bit: scale of a token
  int16_t* token;     // [P] token of row r
  int16_t* id;        // [P] expert of pair (token, slot)
  int16_t* active;    // [E] experts that have rows
  int16_t* first;     // [E + 1] first row of the a-th active expert
};

__device__ __forceinline__ Lists lists_at(uint8_t* p, int P, int E) {
  Lists l;
  l.weight = reinterpret_cast<float*>(p);
  l.pair_weight = l.weight + P;
  l.x_scale = l.pair_weight + P;
  l.token = reinterpret_cast<int16_t*>(l.x_scale + P);
  l.id = l.token + P;
  l.active = l.id + P;
  l.first = l.active + E;
  return l;
}

__host__ inline int lists_bytes(int P, int E) { return (16 * P + 4 * E + 2 + 127) / 128 * 128; }

__device__ __forceinline__ float activate(float g, int act) {
  if (act == FO_ACT_NONE) return g;
  if (act == FO_ACT_RELU) return g > 0.0f ? g : 0.0f;
  // (Not the fast forms: their division gives 0 where 1 + e^-g passes 2^126, though
  // silu is 1e-36 there, and their exponential loses a bit per doubling of g.  They
  // save 0.8% at 48 tokens of 4-bit weights, 346 us of 349, and nothing at 1 or 8.)
  return g / (1.0f + expf(-g));
}

// ------------------------------------------------------------------ router

// Logits of a block of EB experts x 8 tokens by one CTA: its warps share out
// the columns, 256 at a time, and their sums meet in shared memory.
template <int EB>
__device__ void router_block(const FewArgs& a, int e0, int t0, float* red) {
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int nt = min(a.T - t0, 8);
  float acc[EB][8];
#pragma unroll
  for (int e = 0; e < EB; ++e)
#pragma unroll
    for (int t = 0; t < 8; ++t) acc[e][t] = 0.0f;
  for (int k = (warp * 32 + lane) * 8; k < a.H; k += warps * 256) {
    uint4 r[EB], x[8];     // (all loads, then all products)
#pragma unroll
    for (int e = 0; e < EB; ++e)
      r[e] = e0 + e < a.E
                 ? __ldg(reinterpret_cast<const uint4*>(a.router + int64_t(e0 + e) * a.H + k))
                 : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int t = 0; t < 8; ++t)
      x[t] = t < nt ? __ldg(reinterpret_cast<const uint4*>(a.x + (t0 + t) * a.x_stride + k))
                    : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t >= nt) break;
      const uint32_t xw[4] = {x[t].x, x[t].y, x[t].z, x[t].w};
#pragma unroll
      for (int e = 0; e < EB; ++e) {
        const uint32_t rw[4] = {r[e].x, r[e].y, r[e].z, r[e].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[e][t] = fmaf(bf16lo(xw[i]), bf16lo(rw[i]), acc[e][t]);
          acc[e][t] = fmaf(bf16hi(xw[i]), bf16hi(rw[i]), acc[e][t]);
        }
      }
    }
  }
  __syncthreads();   // red is free
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    if (t >= nt) break;
#pragma unroll
    for (int e = 0; e < EB; ++e) {
      float v = acc[e][t];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) red[(e * 8 + t) * warps + warp] = v;
    }
  }
  __syncthreads();
  if (threadIdx.x < EB * 8) {
    const int e = e0 + threadIdx.x / 8, t = threadIdx.x % 8;
    if (e < a.E && t < nt) {
      float v = 0.0f;
      for (int w = 0; w < warps; ++w) v += red[threadIdx.x * warps + w];
      __stcg(a.logits + int64_t(t0 + t) * a.E + e, v);
    }
  }
}

// ------------------------------------------------------------------ f16 with scales

// The scale byte of 32 values kept as f16: with s = the exponent of the
// largest magnitude - 14 they stay below 2^15.
__device__ __forceinline__ uint32_t half_scale(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  if (e == 255u) return 255u;
  return e > 15u ? e - 14u : 1u;
}

__device__ __forceinline__ uint16_t half_value(float v, uint32_t s) {
  if (s == 255u) return 0;   // the block's scale is NaN
  return __half_as_ushort(__float2half_rn(v * __uint_as_float((254u - s) << 23)));
}

// x as f16 with one scale per token, a CTA per token (from the last CTA on: the
// first have the router), zeros past H; and zeros (of scale 1) for h past its
// last block of 32 columns.  `red`: a word per warp.
__device__ void scale_x(const FewArgs& a, uint32_t* red) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  const int from_last = int(gridDim.x) - 1 - int(blockIdx.x);
  for (int t = from_last; t < a.T; t += int(gridDim.x)) {
    const uint16_t* x = a.x + t * a.x_stride;
    uint32_t m = 0;
    for (int c = threadIdx.x * 8; c < a.H; c += blockDim.x * 8) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(x + c));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    __syncthreads();
    if (lane == 0) red[warp] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, lane < warps ? red[lane] : 0u);
    const uint32_t s = half_scale(m << 16);
    for (int c = threadIdx.x * 8; c < a.hp; c += blockDim.x * 8) {
      const uint4 v = c < a.H ? __ldg(reinterpret_cast<const uint4*>(x + c)) : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = half_value(bf16lo(w[i]), s) | uint32_t(half_value(bf16hi(w[i]), s)) << 16;
      *reinterpret_cast<uint4*>(a.xq + (int64_t(c >> 8) * a.T + t) * kMxToken + (c & 255) * 2) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (threadIdx.x == 0)
      a.x_scale[t] = s == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(s << 23);
  }
  const int used = (a.I + 31) / 32 * 32;
  if (used < a.ip)
    for (int r = from_last * warps + warp; r < a.T * a.K; r += int(gridDim.x) * warps)
      for (int c = used + lane; c < a.ip; c += 32) {
        uint8_t* to = a.hq + (int64_t(c >> 8) * a.h_rows + r) * kMxToken;
        reinterpret_cast<uint16_t*>(to)[c & 255] = 0;
        if (lane == 0) reinterpret_cast<float*>(to + 512)[(c & 255) >> 5] = 1.0f;
      }
}

// ------------------------------------------------------------------ work items

// A tile of the first product: hidden rows [i0, i0 + n) of the a-th active
// expert; and the walk over a CTA's granules, tile by tile.
struct HiddenTile {
  int32_t a, i0, n;
};

struct HiddenWalk {
  int32_t left, a, g;
  __device__ __forceinline__ HiddenWalk(int from, int to, int per_expert)
      : left(to - from), a(from / per_expert), g(from % per_expert) {}
  __device__ __forceinline__ bool next(int per_expert, int granule, int I, HiddenTile& t) {
    if (left <= 0) return false;
    const int n = min(min(left, per_expert - g), 64 / granule);
    t.a = a;
    t.i0 = g * granule;
    t.n = min(n * granule, I - t.i0);
    left -= n;
    g += n;
    if (g == per_expert) g = 0, ++a;
    return true;
  }
};

// A run of the second product: output rows of block rb, the a-th active
// expert, stages [k0, k0 + n) of its columns; and the walk over them.
struct OutputRun {
  int32_t rb, a, k0, n;
};

struct OutputWalk {
  int32_t left, rb, a, k;
  __device__ __forceinline__ OutputWalk(int from, int to, int active, int k_stages)
      : left(to - from) {
    const int unit = from / k_stages;
    k = from % k_stages;
    rb = unit / max(active, 1);
    a = unit % max(active, 1);
  }
  __device__ __forceinline__ bool next(int active, int k_stages, OutputRun& r) {
    if (left <= 0) return false;
    r.rb = rb;
    r.a = a;
    r.k0 = k;
    r.n = min(left, k_stages - k);
    left -= r.n;
    k += r.n;
    if (k == k_stages) {
      k = 0;
      if (++a == active) a = 0, ++rb;
    }
    return true;
  }
};

// ------------------------------------------------------------------ instructions

// 16 bytes from global to shared memory, zeros where !valid (src is then not
// read but must be an address).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
               "l"(src), "r"(valid ? 16u : 0u), "l"(policy)
               : "memory");
}
// Arrive on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm2(uint32_t addr, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];"
               : "=r"(r0), "=r"(r1)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// d += a . b for 16 rows, 8 columns, 16 deep; bf16 or f16 operands.
template <bool HALF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (HALF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero, f16 operands.
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Place of 16-byte piece `p` (of a bf16 stage's 16 per row) of row `r` in a
// tile of `rows` rows: two halves of 128 bytes per row, pieces rotated by row
// so that eight rows' same pieces lie in different banks.
__device__ __forceinline__ uint32_t tile_place(int r, int p, int rows) {
  return uint32_t((p >> 3) * rows * 128 + r * 128 + (((p & 7) ^ (r & 7)) << 4));
}

// The same for 4-bit codes: 128 bytes per row, eight pieces of 32 codes, in
// the order of the TMA's 128-byte swizzle.
__device__ __forceinline__ uint32_t code_place(int r, int p) {
  return uint32_t(r * 128 + ((p ^ (r & 7)) << 4));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Among the computing warps.
constexpr int kMathThreads = 256;
__device__ __forceinline__ void math_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kMathThreads) : "memory");
}

// The same, and whether all say yes: these warps give up together, so that none
// is left at a barrier.
__device__ __forceinline__ bool math_all(bool yes) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(out)
      : "r"(uint32_t(yes)), "n"(kMathThreads)
      : "memory");
  return out != 0;
}

// One warp waits (bounded) until the grid's count reaches every CTA.
__device__ __forceinline__ bool wait_grid(const uint32_t* count, uint32_t target,
                                          volatile int* abort_flag, int32_t* status) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) {
    uint64_t t0 = 0;
    for (uint32_t i = 1; ld_acquire_gpu(count) < target; ++i) {
      if (i % 64) continue;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (*abort_flag || now - t0 > kGridWaitNs) {
        *abort_flag = 1;
        atomicCAS(status, 0, int32_t(FO_ERR_TIMEOUT));
        ok = 0;
        break;
      }
    }
  }
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}

// ------------------------------------------------------------------ a stage's products

// bf16: this warp's 16 rows of the stage (8 from lo, 8 from hi on) times nt
// tiles of 8 tokens.  The weights' 16 rows x 128 columns are taken first, then
// two tiles of tokens at a time: eight independent steps' loads, and two chains
// of products (with the columns outermost a step waited for its own loads: 1330
// cycles per stage instead of 740 at 12 tokens).
template <int NT>
__device__ __forceinline__ void stage_bf16(uint32_t stage, int lo, int hi, int nt,
                                           float (&acc)[NT][4]) {
  const int lane = threadIdx.x & 31;
  const int row = ((lane & 8) ? hi : lo) + (lane & 7);
  const uint32_t tokens = stage + 32768;
  const int nb = nt * 8;
  uint32_t w[8][4];
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) ldsm4(stage + tile_place(row, ks * 2 + (lane >> 4), 128), w[ks]);
#pragma unroll
  for (int j = 0; j < NT; j += 2) {
    if (j >= nt) break;
    const int half = (lane >> 3) & 1;
    if (j + 1 < NT && j + 1 < nt) {
      uint32_t t[8][4];
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        ldsm4(tokens + tile_place(j * 8 + (lane >> 4) * 8 + (lane & 7), ks * 2 + half, nb), t[ks]);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        mma16816<false>(acc[j], w[ks][0], w[ks][1], w[ks][2], w[ks][3], t[ks][0], t[ks][1]);
        if constexpr (NT > 1)
          mma16816<false>(acc[j + 1 < NT ? j + 1 : 0], w[ks][0], w[ks][1], w[ks][2], w[ks][3],
                          t[ks][2], t[ks][3]);
      }
    } else {
      uint32_t t[8][2];
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        ldsm2(tokens + tile_place(j * 8 + (lane & 7), ks * 2 + half, nb), t[ks][0], t[ks][1]);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        mma16816<false>(acc[j], w[ks][0], w[ks][1], w[ks][2], w[ks][3], t[ks][0], t[ks][1]);
    }
  }
}

// Four scale bytes as floats.
__device__ __forceinline__ void scales_of(uint32_t w, float (&s)[4]) {
  uint32_t p[2];
  asm("{\n\t.reg .b16 h0, h1;\n\t"
      "mov.b32 {h0, h1}, %2;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %0, h0;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %1, h1;\n\t}"
      : "=r"(p[0]), "=r"(p[1])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 2; ++i) s[2 * i] = bf16lo(p[i]), s[2 * i + 1] = bf16hi(p[i]);
}

// 4-bit: a block of 32 columns is two MMAs.  A thread takes 8 consecutive
// codes of a row (one word) and the same 8 columns of a token (16 bytes); which
// of the MMA's 16 columns they stand in does not matter as long as both agree.
// code: the thread's word of the first block in its first row (those of the
// other blocks differ in the swizzled bits only); its second row is 64 rows
// further in the first product, 8 in the second (SECOND, where the tokens'
// values have a scale per block, too).  scale0, scale1: where the rows' scales
// are; blocks: of the stage's eight, those that exist.
template <int NT, bool SECOND>
__device__ __forceinline__ void stage_mx(uint32_t stage, uint32_t code, uint32_t scale0,
                                         uint32_t scale1, int rows, int blocks,
                                         float (&acc)[NT][4]) {
  constexpr uint32_t kRow1 = SECOND ? 8 * 128 : 64 * 128;
  // blocks whose operands are taken before the first product; with one tile of
  // tokens there are registers for all
  constexpr int kTake = NT == 1 ? 8 : 4;
  const int lane = threadIdx.x & 31, c = lane & 3;
  // rows past the last token's read that one again, which costs nothing (a row of
  // its own for each of the eight: 416 cycles of shared memory per stage)
  const auto token = [&](int i) {
    return stage + kMxTokens + uint32_t(min(i, rows - 1)) * kMxToken;
  };
  code += stage;
  scale0 += stage;
  scale1 += stage;
  // (past the matrix codes and tokens are zeros, scales whatever was there)
  const bool two = blocks > 4;
#pragma unroll
  for (int b0 = 0; b0 < 8; b0 += kTake) {
    uint32_t w0[kTake], w1[kTake];
    float s0[kTake / 4][4], s1[kTake / 4][4];
#pragma unroll
    for (int b = 0; b < kTake; ++b) {
      const uint32_t at = code ^ uint32_t((b0 + b) << 4);
      w0[b] = lds32(at);
      w1[b] = lds32(at + kRow1);
    }
#pragma unroll
    for (int q = 0; q < kTake / 4; ++q) {
      const bool in = b0 / 4 + q == 0 || two;
      scales_of(in ? lds32(scale0 + (b0 / 4 + q) * 512) : 0u, s0[q]);
      scales_of(in ? lds32(scale1 + (b0 / 4 + q) * 512) : 0u, s1[q]);
    }
    // (with more than one tile of tokens the codes are decoded once for all)
    uint32_t p[NT > 1 ? kTake : 1][4], r[NT > 1 ? kTake : 1][4];
    if constexpr (NT > 1) {
#pragma unroll
      for (int b = 0; b < kTake; ++b) {
        mx_decode8(w0[b], p[b]);
        mx_decode8(w1[b], r[b]);
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j * 8 >= rows) break;
      uint32_t t[kTake][4], u0[kTake / 4][4], u1[kTake / 4][4];
#pragma unroll
      for (int b = 0; b < kTake; ++b)
        lds128(token(j * 8 + (lane >> 2)) + c * 16 + (b0 + b) * 64, t[b]);
      if constexpr (SECOND) {
#pragma unroll
        for (int q = 0; q < kTake / 4; ++q) {
          lds128(token(j * 8 + c * 2) + 512 + (b0 / 4 + q) * 16, u0[q]);
          lds128(token(j * 8 + c * 2 + 1) + 512 + (b0 / 4 + q) * 16, u1[q]);
        }
      }
#pragma unroll
      for (int b = 0; b < kTake; ++b) {
        const int at = NT > 1 ? b : 0;
        if constexpr (NT == 1) {
          mx_decode8(w0[b], p[0]);
          mx_decode8(w1[b], r[0]);
        }
        float d[4];
        mma16816_zero(d, p[at][0], r[at][0], p[at][1], r[at][1], t[b][0], t[b][1]);
        mma16816<true>(d, p[at][2], r[at][2], p[at][3], r[at][3], t[b][2], t[b][3]);
        if constexpr (SECOND) {
          uint64_t lo = pack2(d[0], d[1]), hi = pack2(d[2], d[3]);
          const uint64_t u =
              pack2(__uint_as_float(u0[b / 4][b % 4]), __uint_as_float(u1[b / 4][b % 4]));
          unpack2(mul2(lo, u), d[0], d[1]);
          unpack2(mul2(hi, u), d[2], d[3]);
        }
        acc[j][0] = fmaf(d[0], s0[b / 4][b % 4], acc[j][0]);
        acc[j][1] = fmaf(d[1], s0[b / 4][b % 4], acc[j][1]);
        acc[j][2] = fmaf(d[2], s1[b / 4][b % 4], acc[j][2]);
        acc[j][3] = fmaf(d[3], s1[b / 4][b % 4], acc[j][3]);
      }
    }
  }
}

constexpr int kBarBytes = 8 * (2 * kMaxStages) + 16;

// Copying warps and 8 computing warps of 16 rows each.  (With 4-bit weights a
// second set of eight, taking turns at the stages, gives next to nothing: 55 us
// with and without it at 1 token, 144 instead of 147 at 8, 434 instead of 333 at
// 48, where its registers do not suffice.)
constexpr int kThreads = 32 * kCopyWarps + kMathThreads;

// NT: tiles of 8 tokens, at most.
template <bool MX, int NT>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ FewArgs a) {
  constexpr int kCopyThreads = 32 * kCopyWarps;
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint8_t smem_raw[];
  // 1024-byte alignment, for the copies' swizzle
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int P = a.T * a.K;
  const Lists ls = lists_at(smem + a.off_lists, P, a.E);
  float* yacc = reinterpret_cast<float*>(smem + a.off_y);   // [T][kYPitch]; first product: maxima
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + a.off_bar);
  uint64_t* empty = full + kMaxStages;
  int* abort_word = reinterpret_cast<int*>(empty + kMaxStages);
  volatile int* abort_flag = abort_word;
  int* n_active_s = abort_word + 1;
  int* flag_s = abort_word + 2;
  int* most_s = abort_word + 3;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int G = int(gridDim.x), c = int(blockIdx.x);
  constexpr int kGranule = MX ? 32 : 8;     // hidden rows that stay together

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(smem_u32(&full[s]), MX ? kCopyWarps : kCopyThreads);
      mbar_init(smem_u32(&empty[s]), 8);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }

  // ---------------------------------------------------------------- router
  {
    // an expert per CTA while that is one round, else four
    float* red = reinterpret_cast<float*>(smem);
    const int tb = (a.T + 7) / 8, eb = (a.E + 3) / 4;
    if (a.E * tb <= G) {
      if (c < a.E * tb) router_block<1>(a, c % a.E, c / a.E * 8, red);
    } else {
      for (int u = c; u < eb * tb; u += G) router_block<4>(a, u % eb * 4, u / eb * 8, red);
    }
    if constexpr (MX) scale_x(a, reinterpret_cast<uint32_t*>(smem) + 1024);
  }
  // rows of each expert, in the ring's memory until the ring starts
  int32_t* count = reinterpret_cast<int32_t*>(smem + 16384);          // [E]
  for (int e = threadIdx.x; e < a.E; e += kWarps * 32) count[e] = 0;
  __threadfence();
  if constexpr (MX) asm volatile("fence.proxy.async;" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) *flag_s = grid_barrier(a.barrier, uint32_t(G), a.status);
  __syncthreads();
  const bool live = *flag_s != 0;   // every CTA of this launch came to the barrier
  __syncthreads();

  if (live) {
    // ------------------------------------------------------------- choice
    // every CTA makes the same choice from the same logits
    auto choose = [&](auto v) {
      constexpr int V = decltype(v)::value;
      constexpr bool kAhead = V <= 4;     // the next token's logits are under way
      auto load = [&](int t, float (&x)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          x[i] = t < a.T && i * 32 + lane < a.E ? __ldcg(a.logits + int64_t(t) * a.E + i * 32 + lane)
                                                : __int_as_float(0xff800000);
      };
      float x[V], next[V];
      if (kAhead) load(warp, next);
      for (int t = warp; t < a.T; t += kWarps) {
        if (kAhead) {
#pragma unroll
          for (int i = 0; i < V; ++i) x[i] = next[i];
          load(t + kWarps, next);
        } else {
          load(t, x);
        }
        const float x_scale = MX ? __ldcg(a.x_scale + t) : 0.0f;
        int id;
        float w;
        warp_top_k<V>(x, a.E, a.K, a.renormalize != 0, id, w);
        if (lane < a.K) {
          ls.id[t * a.K + lane] = int16_t(id);
          ls.pair_weight[t * a.K + lane] = w;
          if (id >= 0) atomicAdd(&count[id], 1);
        }
        if (MX && lane == 0) ls.x_scale[t] = x_scale;
      }
    };
    if (a.E <= 32)
      choose(Const<1>{});
    else if (a.E <= 128)
      choose(Const<4>{});
    else
      choose(Const<32>{});
    __syncthreads();
    if (warp == 0) {
      int rows = 0, active = 0, most = 1;
      for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane;
        const int n = e < a.E ? count[e] : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += v;
        }
        const uint32_t has = __ballot_sync(0xffffffffu, n > 0);
        const int start = rows + sum - n;
        if (n > 0) {
          const int at = active + __popc(has & ((1u << lane) - 1u));
          ls.active[at] = int16_t(e);
          ls.first[at] = int16_t(start);
        }
        if (e < a.E) count[e] = start;
        most = max(most, n);
        rows += __shfl_sync(0xffffffffu, sum, 31);
        active += __popc(has);
      }
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 0) {
        *most_s = most;
        ls.first[active] = int16_t(rows);
        *n_active_s = active;
      }
      __syncwarp();
      for (int p0 = 0; p0 < P; p0 += 32) {   // rows in the order of pairs
        const int p = p0 + lane;
        const int e = p < P ? ls.id[p] : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        if (e >= 0) {
          const int row = count[e] + rank;
          ls.token[row] = int16_t(p / a.K);
          ls.weight[row] = ls.pair_weight[p];
        }
        __syncwarp();
        if (e >= 0 && rank == 0) count[e] += __popc(same);
        __syncwarp();
      }
    }
    // (threads wrote to the ring's memory and to x's copy, bulk copies follow)
    if constexpr (MX) asm volatile("fence.proxy.async;" ::: "memory");
    __syncthreads();

    const int active = *n_active_s;
    // A stage has room for the most tokens that an expert got.
    const int most = *most_s;
    const int stage_bytes =
        ((MX ? kMxTokens + most * kMxToken : 32768 + (most + 7) / 8 * 8 * 256) + 1023) / 1024 * 1024;
    const int stages = min(a.ring_bytes / stage_bytes, kMaxStages);
    const int per_expert = (a.I + kGranule - 1) / kGranule;
    const Cut cut1(active * per_expert, G, a.inverse_g);
    const int k1 = (a.H + kStageK<MX> - 1) / kStageK<MX>;      // stages of a tile of the first product
    const int k2 = (a.I + kStageK<MX> - 1) / kStageK<MX>;
    const int row_blocks = (a.H + 127) / 128;
    const Cut cut2(row_blocks * active * k2, G, a.inverse_g);
    const HiddenWalk walk1(cut1.first(c), cut1.first(c + 1), per_expert);
    const OutputWalk walk2(cut2.first(c), cut2.first(c + 1), active, k2);
    const uint32_t ring = smem_u32(smem);

    if (!MX && warp < kCopyWarps) {
      // ------------------------------------------------------ copies, bf16
      // A thread has rows r0, r0 + 8, ... of a stage, one of the 16 pieces of 16
      // bytes of each.
      const int tid = threadIdx.x;
      const int piece = tid & 15, r0 = tid >> 4;
      const uint32_t place = tile_place(r0, piece, 128);
      const uint64_t once = tc::policy_evict_first(), keep = tc::policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      // The tokens of stage k: nb rows of 256 bytes, 8 at a time, `rows` of them
      // from memory (`src`: this thread's piece of its first row; the others by
      // their token or in order from `base`), columns below `cols`.
      auto send_tokens = [&](uint32_t dst, int nb, int rows, int first, int k, int64_t row_pitch,
                             int cols, const uint16_t* src, const uint16_t* base, bool by_token) {
        const bool in = k * kStageK<MX> + piece * 8 < cols;
        for (int i = r0; i < nb; i += 8) {
          if (i >= 8) {
            const int row = first + min(i, rows - 1);
            src = base + (by_token ? int64_t(ls.token[row]) : int64_t(row)) * row_pitch +
                  k * kStageK<MX> + piece * 8;
          }
          copy16(dst + 32768 + tile_place(i, piece, nb), in ? src : base, in && i < rows, keep);
        }
      };
      HiddenWalk hidden = walk1;
      HiddenTile t;
      while (ok && hidden.next(per_expert, kGranule, a.I, t)) {
        // a stage's rows: the gate's from 0, the up-projection's from 64 on.
        // A thread's addresses advance by a constant from stage to stage.
        const int64_t gate = int64_t(ls.active[t.a]) * a.w1_rows + t.i0;
        const int first = ls.first[t.a], rows = ls.first[t.a + 1] - first;
        const int nb = (rows + 7) / 8 * 8;
        const int64_t pitch = int64_t(a.H) * 2, up = a.I * pitch;   // bytes
        const uint8_t* src = a.w1 + (gate + r0) * pitch + piece * 16;
        const int left = t.n - r0;             // rows from this thread's first on
        const uint16_t* tok =
            a.x + ls.token[first + min(r0, rows - 1)] * a.x_stride + piece * 8;
        for (int k = 0; k < k1; ++k) {
          ok = tc::wait_warp(smem_u32(&empty[stage]), phase ^ 1, abort_flag, a.status);
          if (!ok) break;
          const uint32_t dst = ring + uint32_t(stage * stage_bytes);
          {
            const uint32_t to = dst + place;
            const bool in = k * kStageK<MX> + piece * 8 < a.H;
            const uint8_t* from = in ? src : a.w1;
            const int64_t step = in ? 8 * pitch : 0, half = in ? up : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (i * 8 < left) {
                copy16(to + i * 1024, from, in, once);
                copy16(to + 8192 + i * 1024, from + half, in, once);
                from += step;
              }
            }
          }
          send_tokens(dst, nb, rows, first, k, a.x_stride, a.H, tok, a.x, true);
          copies_arrive(smem_u32(&full[stage]));
          src += 256;
          tok += kStageK<MX>;
          if (++stage == stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // The second product: the weights of the first stages are on their way
      // before the barrier, the tokens follow after it.
      struct Place {
        OutputWalk walk;
        OutputRun r;
        int k;
        bool more;
        const uint8_t* src;      // weights, or a row of h
      };
      const int64_t pitch = int64_t(a.I) * 2;
      auto open = [&](Place& p, bool weights) {
        p.more = p.walk.next(active, k2, p.r);
        p.k = p.r.k0;
        if (!p.more) return;
        if (weights) {
          const int64_t row = int64_t(ls.active[p.r.a]) * a.w2_rows + p.r.rb * 128;
          p.src = a.w2 + (row + r0) * pitch + piece * 16 + int64_t(p.k) * 256;
        } else {
          const int first = ls.first[p.r.a], rows = ls.first[p.r.a + 1] - first;
          p.src = reinterpret_cast<const uint8_t*>(
              a.h + int64_t(first + min(r0, rows - 1)) * a.I + piece * 8 + p.k * kStageK<MX>);
        }
      };
      Place w{walk2, {}, 0, false, nullptr}, v{walk2, {}, 0, false, nullptr};
      open(w, true);
      open(v, false);
      int w_stage = stage, ahead = 0;    // stages whose weights are under way
      uint32_t w_phase = phase;
      auto send_weights = [&]() {
        ok = tc::wait_warp(smem_u32(&empty[w_stage]), w_phase ^ 1, abort_flag, a.status);
        if (!ok) return;
        const uint32_t dst = ring + uint32_t(w_stage * stage_bytes);
        {
          const bool in = w.k * kStageK<MX> + piece * 8 < a.I;
          const uint32_t to = dst + place;
          const uint8_t* from = in ? w.src : a.w2;
          const int64_t step = in ? 8 * pitch : 0;
          const int left = a.H - w.r.rb * 128 - r0;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (i * 8 < left) {
              copy16(to + i * 1024, from, in, once);
              from += step;
            }
          }
        }
        w.src += 256;
        if (++w.k == w.r.k0 + w.r.n) open(w, true);
        ++ahead;
        if (++w_stage == stages) {
          w_stage = 0;
          w_phase ^= 1;
        }
      };
      while (ok && w.more && ahead < stages) send_weights();
      if (ok && v.more) ok = wait_grid(a.barrier + 1, uint32_t(G), abort_flag, a.status);
      while (ok && v.more) {
        if (ahead == 0) send_weights();
        if (!ok) break;
        const int first = ls.first[v.r.a], rows = ls.first[v.r.a + 1] - first;
        send_tokens(ring + uint32_t(stage * stage_bytes), (rows + 7) / 8 * 8, rows, first, v.k,
                    a.I, a.I, reinterpret_cast<const uint16_t*>(v.src), a.h, false);
        copies_arrive(smem_u32(&full[stage]));
        v.src += 256;
        if (++v.k == v.r.k0 + v.r.n) open(v, false);
        --ahead;
        if (++stage == stages) stage = 0;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");   // none is left when the CTA exits
    } else if (MX && warp < kCopyWarps) {
      // ----------------------------------------------------- copies, 4-bit
      // All of a stage comes by bulk copies: codes (boxes of 128 bytes x 64 rows),
      // scales (blocks of 512 bytes as they are kept, two of a row of blocks, the
      // last may be alone), tokens (values and scales in one piece).  To issue one
      // takes a warp 200 to 400 cycles, a stage's seven 1800 (and the four of
      // scales 1100), so four warps share them, two at most in each, and walk the
      // stages by themselves.
      const bool leader = lane == 0;
      const uint64_t once = tc::policy_evict_first(), keep = tc::policy_evict_last();
      const int64_t kb1 = a.hb, kb2 = a.ib;     // blocks of scales in a row of blocks
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      auto begin = [&]() {
        ok = tc::wait_warp(smem_u32(&empty[stage]), phase ^ 1, abort_flag, a.status);
        return ok;
      };
      auto end = [&]() {
        __syncwarp();
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
      };
      HiddenWalk hidden = walk1;
      HiddenTile t;
      while (ok && hidden.next(per_expert, kGranule, a.I, t)) {
        const int gate = int(ls.active[t.a]) * a.w1_rows + t.i0, up = gate + a.I;
        const int first = ls.first[t.a], rows = ls.first[t.a + 1] - first;
        const int gb = ((gate & 127) + t.n + 127) >> 7, ub = ((up & 127) + t.n + 127) >> 7;
        if (warp < 2) {
          // codes of the gate's or of the up-projection's rows, and where those lie
          // in two rows of blocks, the second's scales.  (Rows past the tile's come
          // along in whole boxes; nobody reads them.)
          const CUtensorMap* map = t.n > 32 ? &a.map_w1[1] : &a.map_w1[0];
          const int row = warp ? up : gate;
          const bool two = (warp ? ub : gb) > 1;
          const uint32_t bytes = t.n > 32 ? 8192 : 4096;
          const uint8_t* scales = a.s1 + (int64_t(row >> 7) + 1) * kb1 * 512;
          for (int k = 0; k < k1 && begin(); ++k, end()) {
            if (leader) {
              const uint32_t sb = !two ? 0 : kb1 - 2 * k > 1 ? 1024 : 512;
              const uint32_t bar = smem_u32(&full[stage]);
              const uint32_t dst = ring + uint32_t(stage * stage_bytes);
              mbar_expect_tx(bar, bytes + sb);
              tc::load_2d(dst + warp * 8192, map, bar, k * 128, row, once);
              if (two) bulk_load_hint(dst + kMxScales + warp * 2048 + 1024, scales, sb, bar, once);
            }
            scales += 1024;
          }
        } else if (warp == 2) {
          const uint8_t* gs = a.s1 + int64_t(gate >> 7) * kb1 * 512;
          const uint8_t* us = a.s1 + int64_t(up >> 7) * kb1 * 512;
          for (int k = 0; k < k1 && begin(); ++k, end()) {
            if (leader) {
              const uint32_t sb = kb1 - 2 * k > 1 ? 1024 : 512, bar = smem_u32(&full[stage]);
              const uint32_t dst = ring + uint32_t(stage * stage_bytes) + kMxScales;
              mbar_expect_tx(bar, 2 * sb);
              bulk_load_hint(dst, gs, sb, bar, once);
              bulk_load_hint(dst + 2048, us, sb, bar, once);
            }
            gs += 1024;
            us += 1024;
          }
        } else {
          const uint8_t* tok0 = a.xq + int64_t(ls.token[first + min(lane, rows - 1)]) * kMxToken;
          const uint8_t* tok1 = a.xq + int64_t(ls.token[first + min(lane + 32, rows - 1)]) * kMxToken;
          const int64_t step = int64_t(a.T) * kMxToken;
          for (int k = 0; k < k1 && begin(); ++k, end()) {
            const uint32_t bar = smem_u32(&full[stage]);
            const uint32_t dst = ring + uint32_t(stage * stage_bytes) + kMxTokens + lane * kMxToken;
            if (leader) mbar_expect_tx(bar, uint32_t(rows * kMxToken));
            __syncwarp();   // (the expected bytes stand before the first that land)
            if (lane < rows) bulk_load_hint(dst, tok0, kMxToken, bar, keep);
            if (lane + 32 < rows) bulk_load_hint(dst + 32 * kMxToken, tok1, kMxToken, bar, keep);
            tok0 += step;
            tok1 += step;
          }
        }
      }
      // The second product: the weights of the first stages are on their way
      // before the barrier, the tokens follow after it.
      if (ok && warp == 3 && walk2.left > 0) {
        ok = wait_grid(a.barrier + 1, uint32_t(G), abort_flag, a.status);
        asm volatile("fence.proxy.async;" ::: "memory");   // h was written by threads
      }
      OutputWalk out = walk2;
      OutputRun r;
      while (ok && out.next(active, k2, r)) {
        const int row = int(ls.active[r.a]) * a.w2_rows + r.rb * 128;
        const int first = ls.first[r.a], rows = ls.first[r.a + 1] - first;
        if (warp < 2) {
          for (int k = r.k0; k < r.k0 + r.n && begin(); ++k, end())
            if (leader) {
              mbar_expect_tx(smem_u32(&full[stage]), 8192);
              tc::load_2d(ring + uint32_t(stage * stage_bytes + warp * 8192), &a.map_w2,
                          smem_u32(&full[stage]), k * 128, row + warp * 64, once);
            }
        } else if (warp == 2) {
          const uint8_t* src = a.s2 + (int64_t(row >> 7) * kb2 + 2 * r.k0) * 512;
          for (int k = r.k0; k < r.k0 + r.n && begin(); ++k, end()) {
            if (leader) {
              const uint32_t sb = kb2 - 2 * k > 1 ? 1024 : 512, bar = smem_u32(&full[stage]);
              mbar_expect_tx(bar, sb);
              bulk_load_hint(ring + uint32_t(stage * stage_bytes) + kMxScales, src, sb, bar, once);
            }
            src += 1024;
          }
        } else {
          const uint8_t* src = a.hq + (int64_t(r.k0) * a.h_rows + first) * kMxToken;
          const uint32_t bytes = uint32_t(rows * kMxToken);
          for (int k = r.k0; k < r.k0 + r.n && begin(); ++k, end()) {
            if (leader) {
              const uint32_t bar = smem_u32(&full[stage]);
              mbar_expect_tx(bar, bytes);
              bulk_load_hint(ring + uint32_t(stage * stage_bytes) + kMxTokens, src, bytes, bar,
                             keep);
            }
            src += int64_t(a.h_rows) * kMxToken;
          }
        }
      }
      if (!ok) {
        // winding down: copies already issued land before the CTA exits
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < tc::kDrainNs) __nanosleep(1000);
      }
    } else {
      // ---------------------------------------------------------- products
      const int mw = warp - kCopyWarps;
      const int mtid = threadIdx.x - kCopyThreads;
      const int g = lane >> 2, c2 = (lane & 3) * 2;   // row and first column of a thread's sums
      int stage = 0;
      uint32_t phase = 0;
      float acc[NT][4];
      // `n` stages into acc; `work`: this warp's rows exist
      auto products = [&](auto second, int n, int rows, int lo, int hi, uint32_t scale0,
                          uint32_t scale1, int blocks, bool work) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
        const uint32_t code = code_place(lo + g, 0) + (lane & 3) * 4;   // 4-bit
        bool ok = true;
        for (int k = 0; k < n; ++k) {
          ok = tc::wait_warp(smem_u32(&full[stage]), phase, abort_flag, a.status);
          if (!ok) break;
          if (work) {
            const uint32_t at = ring + uint32_t(stage * stage_bytes);
            if constexpr (MX)
              stage_mx<NT, decltype(second)::value != 0>(at, code, scale0, scale1, rows,
                                                         blocks - 8 * k, acc);
            else
              stage_bf16<NT>(at, lo, hi, (rows + 7) / 8, acc);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&empty[stage]));
          if (++stage == stages) {
            stage = 0;
            phase ^= 1;
          }
        }
        return math_all(ok);
      };
      bool ok = true;
      HiddenWalk hidden = walk1;
      HiddenTile t;
      while (ok && hidden.next(per_expert, kGranule, a.I, t)) {
        const int first = ls.first[t.a], rows = ls.first[t.a + 1] - first;
        const int nb = (rows + 7) / 8 * 8;
        // a 4-bit row's scales: in the blocks of the tile's gate or up rows
        const int p = mw * 8 + g;                 // this thread's hidden row
        const int gr = (t.i0 & 127) + p, ur = ((t.i0 + a.I) & 127) + p;
        ok = products(Const<0>{}, k1, rows, mw * 8, 64 + mw * 8,
                      kMxScales + (gr >> 7) * 1024 + mx_scale_row(gr & 127),
                      kMxScales + 2048 + (ur >> 7) * 1024 + mx_scale_row(ur & 127),
                      (a.H + 31) / 32, mw * 8 < t.n);
        if (!ok) break;
        float h[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (j * 8 >= nb) break;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if constexpr (MX) {   // the token's scale
              const int i = min(j * 8 + c2 + e, rows - 1);
              const float u = ls.x_scale[ls.token[first + i]];
              acc[j][e] *= u;
              acc[j][e + 2] *= u;
            }
            h[j][e] = p < t.n ? activate(acc[j][e], a.act) * acc[j][e + 2] : 0.0f;
          }
        }
        if constexpr (MX) {
          // 32 hidden rows, those of four warps, share a scale
          uint32_t* top = reinterpret_cast<uint32_t*>(yacc);   // [8 warps][nb]
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (j * 8 >= nb) break;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t m = __float_as_uint(h[j][e]) & 0x7fffffffu;
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
              if (g == 0) top[mw * nb + j * 8 + c2 + e] = m;
            }
          }
          math_sync();
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (j * 8 >= nb) break;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int i = j * 8 + c2 + e;
              if (i >= rows) continue;
              const uint32_t* m = top + (mw & 4) * nb + i;
              const uint32_t s = half_scale(max(max(m[0], m[nb]), max(m[2 * nb], m[3 * nb])));
              const int64_t row = first + i;
              if ((mw & 4) * 8 < t.n) {           // (a whole block, zeros past I)
                const int col = t.i0 + p;
                uint8_t* to = a.hq + (int64_t(col >> 8) * a.h_rows + row) * kMxToken;
                reinterpret_cast<uint16_t*>(to)[col & 255] = half_value(h[j][e], s);
                if ((mw & 3) == 0 && g == 0)
                  reinterpret_cast<float*>(to + 512)[(col & 255) >> 5] =
                      s == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(s << 23);
              }
            }
          }
        } else if (p < t.n) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (j * 8 >= nb) break;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int i = j * 8 + c2 + e;
              if (i < rows)
                reinterpret_cast<__nv_bfloat16*>(a.h)[int64_t(first + i) * a.I + t.i0 + p] =
                    __float2bfloat16_rn(h[j][e]);
            }
          }
        }
      }
      // this CTA's hidden values are written
      if constexpr (MX) asm volatile("fence.proxy.async;" ::: "memory");
      math_sync();
      if (mtid == 0) {     // (a release: what stood before the barrier above is in it)
        uint32_t old;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                     : "=r"(old)
                     : "l"(a.barrier + 1)
                     : "memory");
      }
      OutputWalk out = walk2;
      OutputRun r;
      int rb = -1;                         // the block being summed
      // four sums of a token (32 fours per token)
      auto sums_at = [&](int i) {
        return reinterpret_cast<const float4*>(yacc + (i >> 5) * kYPitch) + (i & 31);
      };
      auto flush = [&]() {
        math_sync();
        // the CTAs that share block rb
        const int lo = rb * active * k2, hi = lo + active * k2;
        const int c0 = cut2.owner(lo), c1 = cut2.owner(hi - 1);
        const bool mine = c0 == c1;
        bool last = mine;
        if (!mine) {
          float* to = a.parts + int64_t(c + rb) * a.T * 128;
          for (int i = mtid; i < a.T * 32; i += kMathThreads)
            __stcg(reinterpret_cast<float4*>(to) + i, *sums_at(i));
          math_sync();
          if (mtid == 0) {
            int32_t parts = c1 - c0 + 1;   // less those whose range is empty
            if (cut2.base == 0)
              for (int k = c0; k <= c1; ++k) parts -= cut2.first(k) == cut2.first(k + 1);
            const int32_t old = atom_add_acq_rel_gpu(a.done + rb, 1);
            *flag_s = old + 1 == parts;
            if (old + 1 == parts) a.done[rb] = 0;   // for the next launch
          }
          math_sync();
          last = *flag_s != 0;
        }
        if (last) {
          // four vectors per thread at once: with many tokens and CTAs the parts'
          // latency is what the join takes
          const float4* from = reinterpret_cast<const float4*>(a.parts + int64_t(rb) * a.T * 128);
          constexpr int kAtOnce = 4;
          for (int i0 = mtid; i0 < a.T * 32; i0 += kMathThreads * kAtOnce) {
            float4 v[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
              const int i = i0 + u * kMathThreads;
              v[u] = mine && i < a.T * 32 ? *sums_at(i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            if (!mine) {
#pragma unroll 4
              for (int k = c0; k <= c1; ++k) {
                const bool has = cut2.base > 0 || cut2.first(k) < cut2.first(k + 1);
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) {
                  const int i = i0 + u * kMathThreads;
                  const float4 x = has && i < a.T * 32 ? __ldcg(from + int64_t(k) * a.T * 32 + i)
                                                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                  v[u].x += x.x, v[u].y += x.y, v[u].z += x.z, v[u].w += x.w;
                }
              }
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
              const int i = i0 + u * kMathThreads, row = rb * 128 + (i & 31) * 4;
              if (i >= a.T * 32 || row >= a.H) continue;   // (H is a multiple of 8)
              __nv_bfloat16* y =
                  reinterpret_cast<__nv_bfloat16*>(a.y) + (i >> 5) * a.y_stride + row;
              y[0] = __float2bfloat16_rn(v[u].x), y[1] = __float2bfloat16_rn(v[u].y);
              y[2] = __float2bfloat16_rn(v[u].z), y[3] = __float2bfloat16_rn(v[u].w);
            }
          }
        }
        math_sync();   // the sums may be overwritten
      };
      while (ok && out.next(active, k2, r)) {
        if (r.rb != rb) {
          if (rb >= 0) flush();
          rb = r.rb;
          for (int i = mtid; i < a.T * kYPitch; i += kMathThreads) yacc[i] = 0.0f;
        }
        const int first = ls.first[r.a], rows = ls.first[r.a + 1] - first;
        ok = products(Const<1>{}, r.n, rows, mw * 16, mw * 16 + 8,
                      kMxScales + mx_scale_row(mw * 16 + g),
                      kMxScales + mx_scale_row(mw * 16 + 8 + g), (a.I + 31) / 32 - 8 * r.k0,
                      r.rb * 128 + mw * 16 < a.H);   // (and the zeros are set)
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (j * 8 >= rows) break;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = j * 8 + c2 + e;
            if (i >= rows) continue;
            float* to = yacc + ls.token[first + i] * kYPitch + mw * 16 + g;
            const float w = ls.weight[first + i];
            to[0] += w * acc[j][e];
            to[8] += w * acc[j][e + 2];
          }
        }
        __syncwarp();   // another lane may add to the same sum next
      }
      if (ok && rb >= 0) flush();
      if (active == 0) {   // no token has an expert: zeros
        for (int64_t j = int64_t(c) * kMathThreads + mtid; j < int64_t(a.T) * a.H;
             j += int64_t(G) * kMathThreads)
          reinterpret_cast<__nv_bfloat16*>(a.y)[j / a.H * a.y_stride + j % a.H] =
              __float2bfloat16_rn(0.0f);
      }
    }
  }

  __syncthreads();
  if (threadIdx.x == 0) grid_barrier_leave(a.barrier + 2, a.barrier, 2, uint32_t(G));
}

struct Layout {
  int64_t done, logits, h, x_scale, xq, hq, parts, bytes;
  int hp, ip, row_blocks;
};

Layout layout_of(const fo_moe_few_desc& d) {
  Layout l{};
  const int64_t pairs = int64_t(d.tokens) * d.top_k;
  l.hp = int(mx_up(d.hidden, kStageK<true>));
  l.ip = int(mx_up(d.inter, kStageK<true>));
  l.row_blocks = int(mx_up(d.hidden, 128) / 128);
  int64_t at = 256;
  auto take = [&](int64_t bytes) {
    const int64_t from = at;
    at += mx_up(bytes, 256);
    return from;
  };
  // the counters' place must not depend on the shape: calls of any shape share
  // a workspace and leave the counters at zero
  l.done = take(4 * kMaxRowBlocks);
  l.logits = take(4 * int64_t(d.tokens) * d.experts);
  if (d.weights == FO_TYPE_BF16) {
    l.h = take(2 * pairs * d.inter);
  } else {
    l.x_scale = take(4 * int64_t(d.tokens));
    l.xq = take(int64_t(d.tokens) * (l.hp / kStageK<true>) * kMxToken);
    l.hq = take(pairs * (l.ip / kStageK<true>) * kMxToken);
  }
  l.parts = take(4 * int64_t(kMaxCtas + l.row_blocks) * d.tokens * 128);
  l.bytes = at;
  return l;
}

template <bool MX, int NT>
fo_status launch(const FewArgs& a, int grid, int smem, cudaStream_t st) {
  static std::once_flag once[64];
  static cudaError_t err[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FO_ERR_CUDA;
  const int slot = dev < 64 ? dev : 63;
  std::call_once(once[slot], [&] {
    err[slot] = cudaFuncSetAttribute(few_kernel<MX, NT>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  });
  if (err[slot] != cudaSuccess) return FO_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, few_kernel<MX, NT>, a) != cudaSuccess) {
    cudaGetLastError();
    return FO_ERR_CUDA;
  }
  return FO_OK;
}

template <bool MX>
fo_status launch_n(const FewArgs& a, int grid, int smem, cudaStream_t st) {
  if (a.T <= 8) return launch<MX, 1>(a, grid, smem, st);
  if (a.T <= 16) return launch<MX, 2>(a, grid, smem, st);
  if (a.T <= 32) return launch<MX, 4>(a, grid, smem, st);
  return launch<MX, 8>(a, grid, smem, st);
}

}  // namespace

int64_t few_workspace_bytes(const fo_moe_few_desc& d) { return layout_of(d).bytes; }

fo_status launch_moe_few(const fo_moe_few_desc& d, const void* x, int64_t x_stride,
                         const void* router, const void* W1, const void* S1, const void* W2,
                         const void* S2, void* y, int64_t y_stride, void* workspace,
                         int32_t* dev_status, void* stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FO_ERR_CUDA;
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  const bool mx = d.weights == FO_TYPE_MX4;
  const Layout l = layout_of(d);
  if (l.row_blocks > kMaxRowBlocks) return FO_ERR_UNSUPPORTED;
  // (weights of more than 2^31 items do not fit any memory; see Cut)
  const int64_t most = int64_t(d.tokens) * d.top_k < d.experts ? d.tokens * d.top_k : d.experts;
  if (most * (int64_t(d.inter) / 8 + 1) > 0x7fffffff ||
      most * l.row_blocks * (int64_t(d.inter) / 128 + 1) > 0x7fffffff)
    return FO_ERR_UNSUPPORTED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  FewArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.x_stride = x_stride;
  a.router = static_cast<const uint16_t*>(router);
  a.w1 = static_cast<const uint8_t*>(W1);
  a.w2 = static_cast<const uint8_t*>(W2);
  a.s1 = static_cast<const uint8_t*>(S1);
  a.s2 = static_cast<const uint8_t*>(S2);
  a.y = static_cast<uint16_t*>(y);
  a.y_stride = y_stride;
  a.T = d.tokens, a.H = d.hidden, a.I = d.inter, a.E = d.experts, a.K = d.top_k;
  a.renormalize = d.renormalize;
  a.act = d.act;
  a.w1_rows = mx ? int(mx_up(2 * int64_t(d.inter), 128)) : 2 * d.inter;
  a.w2_rows = mx ? l.row_blocks * 128 : d.hidden;
  a.barrier = reinterpret_cast<uint32_t*>(ws);
  a.done = reinterpret_cast<int32_t*>(ws + l.done);
  a.logits = reinterpret_cast<float*>(ws + l.logits);
  a.h = reinterpret_cast<uint16_t*>(ws + l.h);
  a.x_scale = reinterpret_cast<float*>(ws + l.x_scale);
  a.xq = ws + l.xq, a.hq = ws + l.hq;
  a.h_rows = d.tokens * d.top_k;
  a.hp = l.hp, a.ip = l.ip;
  a.hb = int(mx_up(d.hidden, 128) / 128), a.ib = int(mx_up(d.inter, 128) / 128);
  a.parts = reinterpret_cast<float*>(ws + l.parts);
  a.status = dev_status;
  const int lists = lists_bytes(d.tokens * d.top_k, d.experts);
  const int y_bytes = int(mx_up(d.tokens * kYPitch * 4, 128));   // the outputs' sums
  const int tail = lists + y_bytes + kBarBytes + 1024;
  a.ring_bytes = (kSmemLimit - tail) / 1024 * 1024;
  // two stages at least, if one expert gets all tokens
  const int64_t largest = mx_up(mx ? kMxTokens + d.tokens * kMxToken
                                   : 32768 + mx_up(d.tokens, 8) * 256, 1024);
  if (a.ring_bytes < 2 * largest) return FO_ERR_UNSUPPORTED;
  a.inverse_g = uint32_t(((1 << 24) + grid - 1) / grid);
  a.off_lists = a.ring_bytes;
  a.off_y = a.off_lists + lists;
  a.off_bar = a.off_y + y_bytes;
  const int smem = a.off_bar + kBarBytes + 1024;
  const auto box = [&](CUtensorMap* map, const void* base, int rows, int blocks, uint32_t height) {
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, uint64_t(blocks) * 64,
                             uint64_t(rows) * d.experts, uint64_t(blocks) * 64, 128, height,
                             CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (mx && (!box(&a.map_w1[0], W1, a.w1_rows, a.hb, 32) ||
             !box(&a.map_w1[1], W1, a.w1_rows, a.hb, 64) ||
             !box(&a.map_w2, W2, a.w2_rows, a.ib, 64)))
    return FO_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return mx ? launch_n<true>(a, grid, smem, st) : launch_n<false>(a, grid, smem, st);
}

}  // namespace fo
