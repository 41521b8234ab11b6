// The balanced router's choice for one token, by one warp.
//
//   s = sigmoid(l) or softmax(l),  c = s + bias           (c decides the choice)
//   a group's score: the sum of its one or two largest c; the top_groups best stay
//   the top_k largest c of what stays; weight = scale s [/ sum of the chosen s]
//
// Two c may be nearer to each other than fp32 tells, and then another choice
// than the mathematics' would follow.  So every decision looks at its margin:
// where it is below what the values may be off, it is made again in fp64 (one
// token in a few thousand on spread-out logits).  Without a bias c grows with l,
// and the logits decide.
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

// What two fp32 choices may be off together.  sigmoid by __expf (2 + 1.173 |l|
// ulp, where s (1 - s) |l| is at most 0.28) and a division of 2 ulp: each below
// 2^-21.  softmax: l - max rounded, __expf, a sum of up to 64 + 5 roundings: below
// 2^-17 of the value.  The addition's rounding.  `ulps`: what a key leaves out.
__device__ __forceinline__ float choice_margin(bool sigmoid, float c, float ulps) {
  return (sigmoid ? 0x1p-20f : 0x1p-16f) + fabsf(c) * (0x1p-22f + ulps * 0x1p-23f);
}

__device__ __forceinline__ float score_32(const ScoreArgs& a, float l, float top, float inv) {
  return a.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-l)) : __expf(l - top) * inv;
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

// The groups that stay, in fp64: bit g of the result.  Of each group only the
// experts that may be among its two largest are computed: those within a margin of
// its second (or only) fp32 choice, `low`, on the lanes of its group.
__device__ __noinline__ uint32_t groups_64(const ScoreArgs& a, int64_t at, int width, float top,
                                           float inv, float low) {
  const int lane = threadIdx.x & 31, lanes = 1 << a.lane_bits;
  const int g = lane >> a.lane_bits, sub = lane & (lanes - 1);
  const bool alike = all_alike(a, at);
  const double sum = a.sigmoid ? 1.0 : softmax_sum_64(a, at, top);
  const float from = low - choice_margin(a.sigmoid, low, 0.0f);
  double m1 = 0.0, m2 = 0.0;
  int n = 0;              // of the two, how many there are
  bool nan = false;       // ranks the group above every number
  for (int i = 0; i < width; ++i) {
    const int k = sub * width + i;
    if (g >= a.groups || k >= a.per) continue;
    const float l = logit_at(a, at + g * a.per + k);
    const float b = a.bias ? __ldg(a.bias + g * a.per + k) : 0.0f;
    const float c = score_32(a, l, top, inv) + b;
    if (l == __int_as_float(0xff800000) || c == __int_as_float(0xff800000) || c < from) continue;
    const double v = alike ? 0.0 : choice_64(a, l, b, top, sum);
    if (v != v) {
      nan = true;
    } else if (n == 0 || v > m1) {
      m2 = m1;
      m1 = v;
      n = n ? 2 : 1;
    } else if (n == 1 || v > m2) {
      m2 = v;
      n = 2;
    }
  }
  for (int o = 1; o < lanes; o <<= 1) {
    const double v1 = shfl_xor_64(m1, o), v2 = shfl_xor_64(m2, o);
    const int k = __shfl_xor_sync(0xffffffffu, n, o);
    nan |= __shfl_xor_sync(0xffffffffu, int(nan), o) != 0;
    if (k == 0) continue;
    if (n == 0) {
      m1 = v1, m2 = v2, n = k;
      continue;
    }
    // the two largest of m1 >= m2 and v1 >= v2
    double next = fmin(m1, v1);
    if (v1 > m1) {
      if (k == 2 && v2 > next) next = v2;
    } else if (n == 2 && m2 > next) {
      next = m2;
    }
    m1 = fmax(m1, v1), m2 = next, n = 2;
  }
  const bool any = g < a.groups && (n > 0 || nan);
  const double score = a.group_top == 2 && n == 2 ? m1 + m2 : m1;
  int rank = 0;
  uint32_t kept = 0;
  for (int h = 0; h < a.groups; ++h) {
    const int from_lane = h << a.lane_bits;
    const double v = __shfl_sync(0xffffffffu, score, from_lane);
    const bool has = __shfl_sync(0xffffffffu, int(any), from_lane) != 0;
    const bool its = __shfl_sync(0xffffffffu, int(nan), from_lane) != 0;
    const bool above = its || nan ? its && (!nan || h < g) : v > score || (v == score && h < g);
    if (has && (!any || above)) ++rank;
  }
  const uint32_t ballot = __ballot_sync(0xffffffffu, any && rank < a.top_groups && sub == 0);
  for (int h = 0; h < a.groups; ++h) kept |= (ballot >> (h << a.lane_bits) & 1u) << h;
  return kept;
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
    const uint32_t from = finite ? order_key(c - choice_margin(a.sigmoid, c, 0.0f)) : best;
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
  double mine = a.bias ? choice_64(a, l, b, top, sum) : double(l);
  // NaN above infinity above the rest, and all of them comparable
  if (mine > 1e300) mine = 1e300;
  if (mine != mine) mine = 1e301;
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const double v = __shfl_sync(0xffffffffu, mine, j);
    const int e = __shfl_sync(0xffffffffu, id, j);
    rank += v > mine || (v == mine && e < id);
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
      return a.bias && i < count ? __ldg(a.bias + first + i) : 0.0f;
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

// The choice for the token whose logits start at `at` and are x: lane j < top_k
// returns slot j in id (-1: none) and weight.
template <int V>
__device__ __forceinline__ void warp_choose(const ScoreArgs& a, const LaneExperts<V>& own,
                                            int64_t at, const float (&x)[V], int& id,
                                            float& weight) {
  const int lane = threadIdx.x & 31;
  const float ninf = __int_as_float(0xff800000);
  constexpr uint32_t kMask = V - 1;
  // softmax's statistics in fp32
  float top = 0.0f, sum = 1.0f;
  if (!a.sigmoid) {
    top = ninf;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, x[i]);
    top = warp_most(top);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += x[i] != ninf ? expf(x[i] - top) : 0.0f;
    sum = warp_add(sum);
  }
  const float inv = 1.0f / sum;
  // keys of the choice; the group's two largest values' keys
  const bool by_logit = a.bias == nullptr;
  const bool exact_groups = by_logit && a.group_top == 1;
  uint32_t key[V], k1 = 0, k2 = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float c = x[i];
    uint32_t k;
    if (!by_logit) {
      c = score_32(a, x[i], top, inv) + own.bias_of(a, i);
      if (x[i] == ninf) c = ninf;
    }
    k = order_key(c);
    key[i] = k >= kLeastKey ? (k & ~kMask) | (kMask - uint32_t(i)) : 0u;
    if (a.groups > 1) {
      if (by_logit && !exact_groups && k >= kLeastKey) k = order_key(score_32(a, x[i], top, inv));
      if (k < kLeastKey) k = 0u;
      k2 = max(k2, min(k1, k));
      k1 = max(k1, k);
    }
  }
  bool open = own.count > 0;
  if (a.groups > 1) {
    const int lanes = 1 << a.lane_bits, g = lane >> a.lane_bits;
    for (int o = 1; o < lanes; o <<= 1) {
      const uint32_t v1 = __shfl_xor_sync(0xffffffffu, k1, o);
      const uint32_t v2 = __shfl_xor_sync(0xffffffffu, k2, o);
      k2 = max(max(k2, v2), min(k1, v1));
      k1 = max(k1, v1);
    }
    uint32_t score = k1;
    if (a.group_top == 2 && k2 != 0u) score = order_key(order_value(k1) + order_value(k2));
    int rank = 0;
#pragma unroll 8
    for (int h = 0; h < a.groups; ++h) {
      const uint32_t v = __shfl_sync(0xffffffffu, score, h << a.lane_bits);
      rank += v > score || (v == score && h < g);
    }
    bool stays = g < a.groups && score != 0u && rank < a.top_groups;
    if (!exact_groups) {
      const uint32_t in = __reduce_min_sync(0xffffffffu, stays ? score : 0xffffffffu);
      const uint32_t out = __reduce_max_sync(0xffffffffu, g < a.groups && !stays ? score : 0u);
      const float vi = order_value(in), vo = order_value(out);
      // (a sum of two is off by twice as much)
      if (out != 0u && (in == out || vi - vo < 2.0f * choice_margin(a.sigmoid, vi, 0.0f))) {
        const float low = a.group_top == 2 && k2 != 0u ? order_value(k2) : order_value(k1);
        const uint32_t kept = groups_64(a, at, V, top, inv, k1 != 0u ? low : ninf);
        stays = g < a.groups && (kept >> g & 1u);
      }
    }
    open = open && stays;
    if (!stays) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = 0u;
    }
  }
  sort_keys<V>(key);
  // the slots and the expert that comes next, for its margin; and on while ranks
  // are too near to tell
  const int K = a.top_k;
  id = -1;
  uint32_t mine = 0u, last = 0u;
  int s = 0;
  const auto round = [&]() {
    const uint32_t head = key[0] & ~kMask;
    const uint32_t best = __reduce_max_sync(0xffffffffu, head);
    if (best == 0u) return false;
    const int win = __ffs(__ballot_sync(0xffffffffu, head == best)) - 1;
    const uint32_t full = __shfl_sync(0xffffffffu, key[0], win);
    if (lane == s) {
      id = (win >> a.lane_bits) * a.per + (win & ((1 << a.lane_bits) - 1)) * V +
           int(kMask - (full & kMask));
      mine = best;
    }
    if (lane == win) {
#pragma unroll
      for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
      key[V - 1] = 0u;
    }
    last = best;
    ++s;
    return true;
  };
  const int rounds = K < 32 ? K + 1 : 32;
  bool more = true;
  while (s < rounds && more) more = round();
  float l = id >= 0 ? logit_at(a, at + id) : 0.0f;
  // (bf16 logits keep all their bits in a key: without a bias they are exact)
  if (!(by_logit && a.bf16)) {
    float b = id >= 0 && a.bias ? __ldg(a.bias + id) : 0.0f;
    const auto near = [&](uint32_t hi, uint32_t lo) {
      if (hi == 0u || lo == 0u) return false;
      if (by_logit || hi == lo) return hi == lo;
      const float c = order_value(hi);
      return c - order_value(lo) < choice_margin(a.sigmoid, c, float(kMask));
    };
    const uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
    const float next_l = __shfl_down_sync(0xffffffffu, l, 1);
    const float next_b = __shfl_down_sync(0xffffffffu, b, 1);
    // (alike neighbours lie in order; but at the last slot another expert may be as
    // near behind them)
    const bool alike = lane + 1 < K && l == next_l && b == next_b;
    const bool unsure = lane < K && lane < 31 && !alike && near(mine, next);
    // (no lane holds the expert after slot 31)
    bool all = false;
    if (K == 32)
      all = near(__shfl_sync(0xffffffffu, mine, 31),
                 __reduce_max_sync(0xffffffffu, key[0] & ~kMask));
    if (__any_sync(0xffffffffu, unsure) || all) {
      // the ranks that follow, as far as they are near to the one before
      bool chain = near(__shfl_sync(0xffffffffu, mine, K - 1), last) && s == K + 1;
      while (chain && s < 32) {
        const uint32_t before = last;
        if (!round()) break;
        chain = near(before, last);
      }
      all |= chain && s == 32;
      if (all) {
        if (!all_alike(a, at)) id = choose_among_all(a, at, V, top, inv, open);
      } else {
        l = id >= 0 ? logit_at(a, at + id) : 0.0f;
        b = id >= 0 && a.bias ? __ldg(a.bias + id) : 0.0f;
        const uint32_t lanes = __ballot_sync(0xffffffffu, id >= 0);
        id = rank_again(a, at, top, id, l, b, __popc(lanes));
      }
      if (lane >= K) id = -1;
      l = id >= 0 ? logit_at(a, at + id) : 0.0f;
    }
  }
  if (lane >= K) id = -1;
  // the weights, in fp32.  Chosen scores may all be far below 1: those to be
  // renormalised share a factor that makes the largest about 1.
  float w = 0.0f;
  if (a.renormalize) {
    const float most = warp_most(id >= 0 ? l : ninf);
    if (id >= 0) {
      if (a.sigmoid) {
        // e^(l - m) / (1 + e^l) with m the largest chosen logit, where that is negative
        const float m = fminf(most, 0.0f);
        w = l < 0.0f ? expf(l - m) / (1.0f + expf(l)) : 1.0f / (1.0f + expf(-l));
      } else {
        // softmax over the chosen, whatever share of the whole they have (a NaN or
        // +inf anywhere enters every score)
        w = sum == sum ? expf(l - most) : sum;
      }
    }
    const float total = warp_add(w);
    w = id >= 0 ? w / total : 0.0f;
  } else if (id >= 0) {
    w = a.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - top) / sum;
  }
  weight = id >= 0 ? a.scale * w : 0.0f;
}

}  // namespace fo
