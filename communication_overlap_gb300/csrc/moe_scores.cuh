// The balanced router's choice for one token, by one warp.
//
//   s = sigmoid(l) or softmax(l),  c = s + bias           (c decides the choice)
//   a group's score: the sum of its one or two largest c; the top_groups best stay
//   the top_k largest c of what stays; weight = scale s [/ sum of the chosen s]
//
// Two c may be nearer to each other than fp32 tells, and then another choice
// than the mathematics' would follow.  So every decision looks at its margin:
// where it is below what the values may be off, it is made again in fp64 (of
// 16384 tokens of 256 experts in 8 groups, normal logits, some 30).  Without a
// bias c grows with l, and the logits decide.
//
// A lane holds V consecutive experts, 2^n lanes a group, as order-preserving keys
// whose lowest bits say which of the lane's experts it is.  So sorting a lane's
// keys is min and max alone, a round of the choice takes the largest head of 32
// sorted lists with one reduction, and the lowest lane that has it is the lowest
// expert.  What those bits cost in precision is part of the margin.
#pragma once

#include <cstdint>

#include "moe_common.cuh"

namespace fo {

struct ScoreArgs {
  const void* logits;
  int64_t stride;
  const float* bias;        // NULL: none
  int32_t bf16, experts, top_k, renormalize;
  int32_t sigmoid;          // else softmax
  int32_t groups, top_groups, group_top;
  int32_t per;              // experts of a group
  int32_t lane_bits;        // a group has 2^lane_bits lanes
  int32_t vec;              // a lane's logits lie on 16 bytes
  float scale;
};

constexpr uint32_t kLeastKey = 0x00800000u;     // of a number; -inf lies below

__device__ __forceinline__ float logit_at(const ScoreArgs& a, int64_t i) {
  return a.bf16 ? __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t*>(a.logits) + i)) << 16)
                : __ldg(static_cast<const float*>(a.logits) + i);
}

// Order-preserving key: larger value, larger key; +0 and -0 equal; NaN (which the
// addition makes positive) above everything, -inf below kLeastKey.
__device__ __forceinline__ uint32_t order_key(float x) {
  const int32_t b = __float_as_int(x + 0.0f);
  return uint32_t(b) ^ (uint32_t(b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// The same in 64 bits, 0 below every number; a NaN above them.
__device__ __forceinline__ uint64_t order_key_64(double x) {
  const int64_t b = __double_as_longlong(x + 0.0);
  return x != x ? ~uint64_t(0) : uint64_t(b) ^ (uint64_t(b >> 63) | uint64_t(1) << 63);
}
__device__ __forceinline__ double order_value_64(uint64_t key) {
  return __longlong_as_double(int64_t(key >> 63 ? key ^ uint64_t(1) << 63 : ~key));
}
__device__ __forceinline__ uint64_t shfl_64(uint64_t x, int from) {
  return __shfl_sync(0xffffffffu, static_cast<unsigned long long>(x), from);
}

__device__ __forceinline__ float warp_add(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float warp_most(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ double shfl_xor_64(double x, int o) {
  return __shfl_xor_sync(0xffffffffu, x, o);
}

// What two fp32 choices may be off together: `score`, for their scores, and what the
// choice's own magnitude adds, the addition's rounding and the `ulps` that a key
// leaves out.
//  sigmoid: the power of two's argument is rounded twice (|l| 2^-23 of the
//      exponential, where s (1 - s) |l| is at most 0.28), ex2.approx is off by 2^-22,
//      the addition by 2^-24, rcp.approx by 2^-23: each below 2^-21.
//  softmax: of a score p, which is at most the largest, 1 / sum: p |l - max| 2^-23 (at
//      most 0.37 2^-23), ex2.approx, rcp.approx, the product, and the sum of expf
//      (2 ulp) with V + 5 roundings: each below (V + 16) 2^-24.
__device__ __forceinline__ float score_margin(bool sigmoid, float inv, int v) {
  return sigmoid ? 0x1p-20f : inv * float(v + 16) * 0x1p-23f;
}
__device__ __forceinline__ float choice_margin(float score, float c, float ulps) {
  return score + fabsf(c) * (0x1p-22f + ulps * 0x1p-23f);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float inverse_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid_32(float l) {
  return inverse_fast(1.0f + exp2_fast(l * -kLog2e));
}
__device__ __forceinline__ float softmax_32(float l, float top, float inv) {
  return exp2_fast((l - top) * kLog2e) * inv;
}
__device__ __forceinline__ float score_32(const ScoreArgs& a, float l, float top, float inv) {
  return a.sigmoid ? sigmoid_32(l) : softmax_32(l, top, inv);
}

// A choice in fp64: top and sum are softmax's, of the token.
__device__ __forceinline__ double choice_64(const ScoreArgs& a, float l, float b, float top,
                                            double sum) {
  const double s = a.sigmoid ? 1.0 / (1.0 + exp(-double(l))) : exp(double(l) - double(top)) / sum;
  return s + double(b);
}

// softmax's sum over the token whose logits start at `at`.
__device__ __noinline__ double softmax_sum_64(const ScoreArgs& a, int64_t at, float top) {
  double v = 0.0;
  for (int e = threadIdx.x & 31; e < a.experts; e += 32)
    v += exp(double(logit_at(a, at + e)) - double(top));      // (-inf: 0)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += shfl_xor_64(v, o);
  return v;
}

// Whether a token's experts are all alike: then every decision goes by index.
__device__ __noinline__ bool all_alike(const ScoreArgs& a, int64_t at) {
  const float l0 = logit_at(a, at), b0 = a.bias ? __ldg(a.bias) : 0.0f;
  bool alike = true;
  for (int e = threadIdx.x & 31; e < a.experts; e += 32)
    if (logit_at(a, at + e) != l0 || (a.bias && __ldg(a.bias + e) != b0)) alike = false;
  return __all_sync(0xffffffffu, alike);
}

// A choice among any number of near ties: each round takes the largest fp32 value
// and decides among those within its margin in fp64, or by index where they are
// alike.  open: this lane's experts may be chosen.  Slot j's expert on lane j.
__device__ __noinline__ int choose_among_all(const ScoreArgs& a, int64_t at, int width, float top,
                                             float inv, bool open) {
  const int lane = threadIdx.x & 31;
  const int first = (lane >> a.lane_bits) * a.per, sub = lane & ((1 << a.lane_bits) - 1);
  const float ninf = __int_as_float(0xff800000), pinf = __int_as_float(0x7f800000);
  const double sum = a.sigmoid ? 1.0 : softmax_sum_64(a, at, top);
  uint64_t taken = 0;
  int mine = -1;
  const auto value = [&](int i, float& l, float& b) {     // -inf: not to be chosen
    const int k = sub * width + i;
    if (!open || k >= a.per || (taken >> i & 1)) return ninf;
    l = logit_at(a, at + first + k);
    b = a.bias ? __ldg(a.bias + first + k) : 0.0f;
    if (l == ninf) return ninf;
    return a.bias ? score_32(a, l, top, inv) + b : l;
  };
  for (int s = 0; s < a.top_k; ++s) {
    uint32_t best = 0;
    float l = 0.0f, b = 0.0f;
    for (int i = 0; i < width; ++i) best = max(best, order_key(value(i, l, b)));
    best = __reduce_max_sync(0xffffffffu, best);
    if (best < kLeastKey) break;
    const float c = order_value(best);
    // (without a bias the values are the logits, and exact; so are infinities and NaN)
    const bool finite = a.bias != nullptr && c < pinf;
    const uint32_t from =
        finite ? order_key(c - choice_margin(score_margin(a.sigmoid, inv, width), c, 0.0f)) : best;
    uint32_t low = 0xffffffffu;       // the lowest candidate
    for (int i = width - 1; i >= 0; --i) {
      const uint32_t k = order_key(value(i, l, b));
      if (k >= from && k >= kLeastKey) low = uint32_t(first + sub * width + i);
    }
    low = __reduce_min_sync(0xffffffffu, low);
    uint32_t pick = low;
    if (finite) {
      const float l0 = logit_at(a, at + low), b0 = __ldg(a.bias + low);
      bool alike = true;
      for (int i = 0; i < width; ++i) {
        const uint32_t k = order_key(value(i, l, b));
        if (k >= from && k >= kLeastKey && (l != l0 || b != b0)) alike = false;
      }
      if (!__all_sync(0xffffffffu, alike)) {
        double most = 0.0;
        uint32_t which = 0xffffffffu;
        for (int i = 0; i < width; ++i) {
          const uint32_t k = order_key(value(i, l, b));
          if (k < from || k < kLeastKey) continue;
          const double v = choice_64(a, l, b, top, sum);
          if (which == 0xffffffffu || v > most) most = v, which = uint32_t(first + sub * width + i);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const double v = shfl_xor_64(most, o);
          const uint32_t e = __shfl_xor_sync(0xffffffffu, which, o);
          if (e != 0xffffffffu &&
              (which == 0xffffffffu || v > most || (v == most && e < which)))
            most = v, which = e;
        }
        pick = which;
      }
    }
    const int i = int(pick) - first - sub * width;
    if (open && i >= 0 && i < width && sub * width + i < a.per) taken |= uint64_t(1) << i;
    if (lane == s) mine = int(pick);
  }
  return mine;
}

// Lanes 0 .. n - 1 hold candidates, the fp32 choice's ranks: they are ranked again
// in fp64, or without a bias by their logits, ties to the lowest expert.
__device__ __noinline__ int rank_again(const ScoreArgs& a, int64_t at, float top, int id, float l,
                                       float b, int n) {
  const int lane = threadIdx.x & 31;
  const double sum = a.sigmoid || !a.bias ? 1.0 : softmax_sum_64(a, at, top);
  const double mine = a.bias ? choice_64(a, l, b, top, sum) : double(l);
  const uint64_t key = order_key_64(mine);
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const uint64_t v = shfl_64(key, j);
    const int e = __shfl_sync(0xffffffffu, id, j);
    rank += v > key || (v == key && e < id);
  }
  int out = -1;
  for (int j = 0; j < n; ++j) {
    const int r = __shfl_sync(0xffffffffu, rank, j), e = __shfl_sync(0xffffffffu, id, j);
    if (r == lane) out = e;
  }
  return out;
}

// Sorts V keys, the largest first (an odd-even merge network).
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2) {
#pragma unroll
    for (int q = p; q >= 1; q /= 2) {
#pragma unroll
      for (int j = q % p; j < V - q; j += 2 * q) {
#pragma unroll
        for (int i = 0; i < q; ++i) {
          if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t hi = max(k[i + j], k[i + j + q]), lo = min(k[i + j], k[i + j + q]);
            k[i + j] = hi, k[i + j + q] = lo;
          }
        }
      }
    }
  }
}

// What a lane holds of every token.
template <int V>
struct LaneExperts {
  int first;          // its first expert
  int count;          // 0 .. V
  float bias[V <= 8 ? V : 1];

  __device__ __forceinline__ LaneExperts(const ScoreArgs& a) {
    const int lane = threadIdx.x & 31;
    const int g = lane >> a.lane_bits, k = (lane & ((1 << a.lane_bits) - 1)) * V;
    first = g * a.per + k;
    count = g < a.groups ? max(0, min(V, a.per - k)) : 0;
    if constexpr (V <= 8) {
#pragma unroll
      for (int i = 0; i < V; ++i) bias[i] = a.bias && i < count ? __ldg(a.bias + first + i) : 0.0f;
    }
  }
  __device__ __forceinline__ float bias_of(const ScoreArgs& a, int i) const {
    if constexpr (V <= 8)
      return bias[i];
    else
      return i < count ? __ldg(a.bias + first + i) : 0.0f;
  }
  // The logits of the token that starts at `at`; -inf past the lane's experts.
  __device__ __forceinline__ void load(const ScoreArgs& a, int64_t at, bool live,
                                       float (&x)[V]) const {
    if (V >= 4 && a.vec) {      // (a lane has all V or none)
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = __int_as_float(0xff800000);
      if (!live || count == 0) return;
      if (a.bf16) {
        if constexpr (V >= 8) {
          const uint4* p =
              reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.logits) + at + first);
#pragma unroll
          for (int i = 0; i < V / 8; ++i) {
            const uint4 w = __ldg(p + i);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) x[8 * i + j] = j & 1 ? bf16hi(u[j / 2]) : bf16lo(u[j / 2]);
          }
        }
      } else {
        const float4* p =
            reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + at + first);
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          const float4 w = __ldg(p + i);
          x[4 * i] = w.x, x[4 * i + 1] = w.y, x[4 * i + 2] = w.z, x[4 * i + 3] = w.w;
        }
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      x[i] = live && i < count ? logit_at(a, at + first + i) : __int_as_float(0xff800000);
  }
};

// One token's choice on its way through warp_choose.
template <int V>
struct Choice {
  uint32_t key[V];
  float top, sum, inv;      // softmax's
  bool open;                // this lane's experts may be chosen
  int win;                  // rank `lane`: the lane that had it, and its key
  uint32_t full;
};

// The keys, sorted.
template <int V>
__device__ __forceinline__ void make_keys(const ScoreArgs& a, const LaneExperts<V>& own,
                                          const float (&x)[V], Choice<V>& c) {
  const float ninf = __int_as_float(0xff800000);
  constexpr uint32_t kMask = V - 1;
  c.top = 0.0f, c.sum = c.inv = 1.0f;
  if (!a.sigmoid) {
    c.top = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) c.top = fmaxf(c.top, x[i]);
    c.top = warp_most(c.top);
    c.sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) c.sum += x[i] != ninf ? expf(x[i] - c.top) : 0.0f;
    c.sum = warp_add(c.sum);
    c.inv = inverse_fast(c.sum);
  }
  float v[V];
  if (a.bias == nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = x[i] + 0.0f;       // (-0 becomes +0)
  } else if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = sigmoid_32(x[i]) + own.bias_of(a, i);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = softmax_32(x[i], c.top, c.inv) + own.bias_of(a, i);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int32_t b = __float_as_int(v[i]);
    const uint32_t k = uint32_t(b) ^ (uint32_t(b >> 31) | 0x80000000u);
    // (a NaN is no -inf; fminf takes the number of the two)
    c.key[i] = fminf(x[i], v[i]) == ninf ? 0u : (k & ~kMask) | (kMask - uint32_t(i));
  }
  sort_keys<V>(c.key);
  c.open = own.count > 0;
}

// What a group's score may be off for the bits that its logits' keys leave out, V ulps
// of l each: p |l| <= p |max| + p |l - max|, the latter at most 0.37 of the largest p.
// (Of a sigmoid, whose s (1 - s) |l| is at most 0.28, the other margins hold that.)
template <int V>
__device__ __forceinline__ float cut_logit_margin(const ScoreArgs& a, const Choice<V>& c, float v) {
  return a.bias || a.sigmoid || a.group_top == 1 || a.bf16
             ? 0.0f
             : (v * fabsf(c.top) + c.inv) * (float(V) * 0x1p-22f);
}

// Which groups stay, as far as fp32 tells.
struct GroupCut {
  uint32_t score;           // of this lane's group
  uint32_t second;          // the least choice that it counts
  uint32_t in;              // the last that stays
  float margin;
  bool stays;
  bool near;                // the first that goes may have to stay instead (of every lane)
};

template <int V>
__device__ __forceinline__ GroupCut cut_groups(const ScoreArgs& a, const Choice<V>& c) {
  constexpr uint32_t kMask = V - 1;
  const int lane = threadIdx.x & 31, lanes = 1 << a.lane_bits, g = lane >> a.lane_bits;
  const bool by_logit = a.bias == nullptr;
  GroupCut r;
  // the two largest of the lane, then of the group
  uint32_t k1 = c.key[0] & ~kMask, k2 = V > 1 ? c.key[V > 1 ? 1 : 0] & ~kMask : 0u;
  if (by_logit && a.group_top == 2) {     // (scores grow with the logits)
    if (k1 != 0u) k1 = order_key(score_32(a, order_value(k1), c.top, c.inv));
    if (k2 != 0u) k2 = order_key(score_32(a, order_value(k2), c.top, c.inv));
  }
  for (int o = 1; o < lanes; o <<= 1) {
    const uint32_t v1 = __shfl_xor_sync(0xffffffffu, k1, o);
    const uint32_t v2 = __shfl_xor_sync(0xffffffffu, k2, o);
    k2 = max(max(k2, v2), min(k1, v1));
    k1 = max(k1, v1);
  }
  const bool two = a.group_top == 2 && k2 != 0u;
  r.score = two ? order_key(order_value(k1) + order_value(k2)) : k1;
  r.second = two ? k2 : k1;
  int rank = 0;
#pragma unroll 8
  for (int h = 0; h < a.groups; ++h) {
    const uint32_t v = __shfl_sync(0xffffffffu, r.score, h << a.lane_bits);
    rank += v > r.score || (v == r.score && h < g);
  }
  r.stays = g < a.groups && r.score != 0u && rank < a.top_groups;
  r.in = __reduce_min_sync(0xffffffffu, r.stays ? r.score : 0xffffffffu);
  const uint32_t out = __reduce_max_sync(0xffffffffu, g < a.groups && !r.stays ? r.score : 0u);
  // (bf16 logits are exact; of fp32 ones the keys leave bits out; sums of two are off
  // by twice as much)
  const bool logits = by_logit && a.group_top == 1;
  const float vi = order_value(r.in);
  r.margin = logits ? 0.0f
                    : 2.0f * choice_margin(score_margin(a.sigmoid, c.inv, V), vi, float(4 * V)) +
                          cut_logit_margin(a, c, vi);
  r.near = out != 0u && (r.in == out ? !(logits && a.bf16) : vi - order_value(out) < r.margin);
  return r;
}

// A sum of two choices of unlike signs is smaller than they are, and off by what they are
// off: the margin counts that, the most of any group (one far from the cut may be off as
// far).  Sums of like signs are near each other only if their choices are as large.
template <int V>
__device__ __noinline__ GroupCut widen_cut(const ScoreArgs& a, GroupCut r) {
  const int g = (threadIdx.x & 31) >> a.lane_bits;
  const float second = order_value(r.second), vi = order_value(r.in);
  // (the larger of the two is the sum without the other; a choice alone is both)
  const float apart =
      g < a.groups && second < 0.0f ? 2.0f * fmaxf(fminf(order_value(r.score) - second, -second), 0.0f)
                                    : 0.0f;
  const float most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(apart)));
  const uint32_t out = __reduce_max_sync(0xffffffffu, g < a.groups && !r.stays ? r.score : 0u);
  r.margin += 2.0f * choice_margin(0.0f, most, float(4 * V));
  r.near = r.near || (out != 0u && vi - order_value(out) < r.margin);
  return r;
}

// The groups near the cut again, in fp64: whether this lane's stays.  Only experts that
// may be among a group's two largest are computed, all of them at once, a lane each: an
// exponential and a division in fp64 take a microsecond.  In the sorted keys of a lane
// they come first.
template <int V>
__device__ __noinline__ bool settle_groups(const ScoreArgs& a, int64_t at, int first, Choice<V> c,
                                           GroupCut r) {
  constexpr uint32_t kMask = V - 1;
  const int lane = threadIdx.x & 31, g = lane >> a.lane_bits;
  // without a bias the largest choice is the largest logit's
  const bool by_logit = a.bias == nullptr, logits = by_logit && a.group_top == 1;
  // groups further than a margin from the last that stays are sure
  const bool unsure = g < a.groups && r.score != 0u &&
                      (r.score == r.in || fabsf(order_value(r.score) - order_value(r.in)) <= r.margin);
  const bool leads = (lane & ((1 << a.lane_bits) - 1)) == 0;
  const int open =
      a.top_groups - __popc(__ballot_sync(0xffffffffu, r.stays && !unsure && leads));
  const float least = order_value(r.second);
  const float low =
      least - (logits ? fabsf(least) * (float(V) * 0x1p-22f)
                      : choice_margin(score_margin(a.sigmoid, c.inv, V), least, float(4 * V)) +
                            cut_logit_margin(a, c, least));
  const double sum = a.sigmoid || logits ? 1.0 : softmax_sum_64(a, at, c.top);
  uint64_t m1 = 0, m2 = 0;      // of group `lane`, the two largest so far
  int mine = -1, held = 0;      // the lane's candidate, and how many lanes have one
  const auto take = [&]() {
    uint64_t key = 0;
    if (mine >= 0) {
      const float l = logit_at(a, at + mine);
      key = order_key_64(logits ? double(l)
                                : choice_64(a, l, a.bias ? __ldg(a.bias + mine) : 0.0f, c.top, sum));
    }
    const int group = mine >= 0 ? mine / a.per : -1;
    for (int j = 0; j < held; ++j) {
      const uint64_t v = shfl_64(key, j);
      const uint64_t k = __shfl_sync(0xffffffffu, group, j) == lane ? v : 0;
      m2 = max(m2, min(m1, k));
      m1 = max(m1, k);
    }
    mine = -1, held = 0;
  };
  for (int i = 0; i < V; ++i) {
    const uint32_t k = c.key[i];
    float v = order_value(k & ~kMask);
    if (by_logit && !logits) v = score_32(a, v, c.top, c.inv);
    const bool in = unsure && k != 0u && !(v < low);
    uint32_t todo = __ballot_sync(0xffffffffu, in);
    if (todo == 0u) break;      // (a lane's keys are sorted)
    if (held + __popc(todo) > 32) take();
    const int e = first + int(kMask - (k & kMask));
    for (; todo; todo &= todo - 1) {
      const int from = __shfl_sync(0xffffffffu, e, __ffs(todo) - 1);
      if (lane == held) mine = from;
      ++held;
    }
  }
  take();
  const uint64_t score = a.group_top == 2 && m2 != 0
                             ? order_key_64(order_value_64(m1) + order_value_64(m2))
                             : m1;
  int rank = 0;
  for (uint32_t todo = __ballot_sync(0xffffffffu, m1 != 0); todo; todo &= todo - 1) {
    const int h = __ffs(todo) - 1;
    const uint64_t v = shfl_64(score, h);
    rank += v > score || (v == score && h < lane);
  }
  const uint32_t best = __ballot_sync(0xffffffffu, m1 != 0 && rank < open);
  return unsure ? (best >> g & 1u) != 0 : r.stays;
}

// The next rank: the largest head of the lanes' lists, on the lowest lane that has
// it.  Its key without the lane's bits, 0 where none is left.
template <int V>
__device__ __forceinline__ uint32_t next_rank(Choice<V>& c, int s) {
  constexpr uint32_t kMask = V - 1;
  const int lane = threadIdx.x & 31;
  const uint32_t head = c.key[0] & ~kMask;
  const uint32_t best = __reduce_max_sync(0xffffffffu, head);
  const int win = __ffs(__ballot_sync(0xffffffffu, head == best)) - 1;
  const uint32_t full = __shfl_sync(0xffffffffu, c.key[0], win);
  c.win = lane == s ? win : c.win;
  c.full = lane == s ? full : c.full;
  const bool mine = lane == win;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t after = i + 1 < V ? c.key[i + 1 < V ? i + 1 : i] : 0u;
    c.key[i] = mine ? after : c.key[i];
  }
  return best;
}

// The choice for N tokens at once, whose logits start at `at` and are x: lane j <
// top_k returns slot j in id (-1: none) and weight.  (Their steps are independent,
// so one's wait for a reduction is filled by the other's.)
template <int V, int N>
__device__ __forceinline__ void warp_choose(const ScoreArgs& a, const LaneExperts<V>& own,
                                            const int64_t (&at)[N], const float (&x)[N][V],
                                            int (&id)[N], float (&weight)[N]) {
  constexpr uint32_t kMask = V - 1;
  const int lane = threadIdx.x & 31, K = a.top_k;
  const bool by_logit = a.bias == nullptr;
  Choice<V> c[N];
#pragma unroll
  for (int n = 0; n < N; ++n) make_keys<V>(a, own, x[n], c[n]);
  if (a.groups > 1) {
    GroupCut r[N];
    bool near = false;
#pragma unroll
    for (int n = 0; n < N; ++n) r[n] = cut_groups<V>(a, c[n]);
    if (a.bias != nullptr && a.group_top == 2) {
      // (a key of a negative number; 0 is none)
      bool unlike = false;
#pragma unroll
      for (int n = 0; n < N; ++n) unlike = unlike || r[n].second - 1u < 0x7fffffffu;
      if (__any_sync(0xffffffffu, unlike)) {
#pragma unroll
        for (int n = 0; n < N; ++n) r[n] = widen_cut<V>(a, r[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) near = near || r[n].near;
    if (near) {
#pragma unroll
      for (int n = 0; n < N; ++n)
        if (r[n].near && !all_alike(a, at[n]))
          r[n].stays = settle_groups<V>(a, at[n], own.first, c[n], r[n]);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      c[n].open = c[n].open && r[n].stays;
#pragma unroll
      for (int i = 0; i < V; ++i) c[n].key[i] = r[n].stays ? c[n].key[i] : 0u;
    }
  }
  // the slots, and the expert that comes next for its margin (bf16 logits alone keep
  // all their bits in a key and need none)
  const bool exact = by_logit && a.bf16;
  const int rounds = exact || K == 32 ? K : K + 1;
  uint32_t last[N];
#pragma unroll
  for (int n = 0; n < N; ++n) c[n].win = 0, c[n].full = 0u;
  for (int s = 0; s < rounds; ++s) {
#pragma unroll
    for (int n = 0; n < N; ++n) last[n] = next_rank<V>(c[n], s);
  }
  uint32_t key[N];    // of rank `lane`
  const auto read = [&](int n) {
    key[n] = c[n].full & ~kMask;
    id[n] = c[n].full == 0u
                ? -1
                : (c[n].win >> a.lane_bits) * a.per + (c[n].win & ((1 << a.lane_bits) - 1)) * V +
                      int(kMask - (c[n].full & kMask));
  };
  float l[N], b[N];
  const auto fetch = [&](int n) {
    l[n] = id[n] >= 0 ? logit_at(a, at[n] + id[n]) : 0.0f;
    b[n] = id[n] >= 0 && !by_logit ? __ldg(a.bias + id[n]) : 0.0f;
  };
#pragma unroll
  for (int n = 0; n < N; ++n) {
    read(n);
    fetch(n);
  }
  if (!exact) {
    const auto near = [&](int n, uint32_t hi, uint32_t lo) {
      if (hi == 0u || lo == 0u) return false;
      if (by_logit || hi == lo) return hi == lo;
      const float v = order_value(hi);
      return v - order_value(lo) < choice_margin(score_margin(a.sigmoid, c[n].inv, V), v, float(V));
    };
    bool unsure[N], all[N], some = false;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t next = __shfl_down_sync(0xffffffffu, key[n], 1);
      const float next_l = __shfl_down_sync(0xffffffffu, l[n], 1);
      const float next_b = __shfl_down_sync(0xffffffffu, b[n], 1);
      // (alike neighbours lie in order; but at the last slot another expert may be as
      // near behind them)
      const bool alike = lane + 1 < K && l[n] == next_l && b[n] == next_b;
      unsure[n] = lane < K && lane < 31 && !alike && near(n, key[n], next);
      all[n] = false;       // (no lane holds the expert after slot 31)
      if (K == 32)
        all[n] = near(n, __shfl_sync(0xffffffffu, key[n], 31),
                      __reduce_max_sync(0xffffffffu, c[n].key[0] & ~kMask));
      some = some || unsure[n] || all[n];
    }
    if (__any_sync(0xffffffffu, some)) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if ((!__any_sync(0xffffffffu, unsure[n]) && !all[n]) || all_alike(a, at[n])) continue;
        // the ranks that follow, as far as they are near to the one before
        int s = rounds;
        bool chain = K < 32 && near(n, __shfl_sync(0xffffffffu, key[n], K - 1), last[n]);
        while (chain && s < 32) {
          const uint32_t before = last[n];
          last[n] = next_rank<V>(c[n], s++);
          chain = near(n, before, last[n]);
        }
        if (all[n] || chain) {
          id[n] = choose_among_all(a, at[n], V, c[n].top, c[n].inv, c[n].open);
        } else {
          read(n);
          fetch(n);
          const uint32_t lanes = __ballot_sync(0xffffffffu, id[n] >= 0);
          id[n] = rank_again(a, at[n], c[n].top, id[n], l[n], b[n], __popc(lanes));
        }
        if (lane >= K) id[n] = -1;
        l[n] = id[n] >= 0 ? logit_at(a, at[n] + id[n]) : 0.0f;
      }
    }
  }
  // the weights, in fp32, by expf and a division of 2 ulp.  Chosen scores may all be
  // far below 1: those to be renormalised share a factor that makes the largest
  // about 1.
  float w[N];
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (lane >= K) id[n] = -1;
  if (a.renormalize) {
    // e^(l - m) / (1 + e^l), m the largest chosen logit where that is negative; softmax
    // over the chosen, whatever share of the whole they have (a NaN or +inf anywhere
    // enters every score)
    float most[N];
#pragma unroll
    for (int n = 0; n < N; ++n)
      most[n] = order_value(__reduce_max_sync(0xffffffffu, id[n] >= 0 ? order_key(l[n]) : 0u));
    if (a.sigmoid) {
#pragma unroll
      for (int n = 0; n < N; ++n)
        w[n] = __fdividef(expf(fminf(l[n], 0.0f) - fminf(most[n], 0.0f)), 1.0f + expf(-fabsf(l[n])));
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) w[n] = c[n].sum == c[n].sum ? expf(l[n] - most[n]) : c[n].sum;
    }
    float sum[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (l[n] != l[n]) w[n] = l[n];       // (fminf would drop a NaN)
      w[n] = id[n] >= 0 ? w[n] : 0.0f;
      sum[n] = w[n];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (o >= K) continue;                // (of lanes without a slot: zeros)
#pragma unroll
      for (int n = 0; n < N; ++n) sum[n] += __shfl_xor_sync(0xffffffffu, sum[n], o);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) w[n] = __fdividef(w[n], sum[n]);
  } else if (a.sigmoid) {
#pragma unroll
    for (int n = 0; n < N; ++n) w[n] = __fdividef(1.0f, 1.0f + expf(-l[n]));
  } else {
#pragma unroll
    for (int n = 0; n < N; ++n) w[n] = __fdividef(expf(l[n] - c[n].top), c[n].sum);
  }
#pragma unroll
  for (int n = 0; n < N; ++n) weight[n] = id[n] >= 0 ? a.scale * w[n] : 0.0f;
}

}  // namespace fo
