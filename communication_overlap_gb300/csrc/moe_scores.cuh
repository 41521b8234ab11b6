// The balanced router's choice for one token, by one warp.
//
//   s = sigmoid(l) or softmax(l),  c = s + bias           (c decides the choice)
//   a group's score: the sum of its one or two largest c; the top_groups best stay
//   the top_k largest c of what stays; weight = scale s [/ sum of the chosen s]
//
// Two c may be nearer to each other than fp32 tells, and then another choice
// than the mathematics' would follow.  So every decision looks at its margin:
// where it is below what the fp32 values may be off, the token is decided again
// in fp64 (one token in a few thousand on spread-out logits).  Without a bias c
// grows with l, and the logits decide, exactly.
#pragma once

#include <cstdint>

#include "moe_common.cuh"

namespace fo {

struct ScoreArgs {
  const float* bias;        // NULL: none
  int32_t sigmoid;          // else softmax
  int32_t groups, top_groups, group_top;
  float scale;
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// What fp32 scores and choices may be off.  sigmoid by __expf (2 + 1.173 |l| ulp,
// and s (1 - s) |l| is at most 0.28) and a division of 2 ulp: below 2^-21.  softmax:
// l - max rounded, __expf, a sum of up to 32 + 5 roundings: below 2^-18 of the
// value.  Both doubled, as two values are compared, and the addition's rounding.
__device__ __forceinline__ float choice_margin(bool sigmoid, float c) {
  return (sigmoid ? 0x1p-20f : 0x1p-17f) + fabsf(c) * 0x1p-22f;
}

// A choice in fp64: top and sum are softmax's, of the token.
__device__ __forceinline__ double choice_64(float l, float b, bool sigmoid, float top,
                                            double sum) {
  const double s = sigmoid ? 1.0 / (1.0 + exp(-double(l))) : exp(double(l) - double(top)) / sum;
  return s + double(b);
}

__device__ __forceinline__ double shfl_xor_64(double x, int o) {
  return __shfl_xor_sync(0xffffffffu, x, o);
}

// softmax's sum; x: V logits per lane, as below.
template <int V>
__device__ __noinline__ double softmax_sum_64(const float* x, int E, float top) {
  double v = 0.0;
  for (int i = 0; i < V; ++i)
    if (i * 32 + int(threadIdx.x & 31) < E) v += exp(double(x[i]) - double(top));   // (-inf: 0)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += shfl_xor_64(v, o);
  return v;
}

// Decided again with fp64 choices: key holds the fp32 keys of the experts that
// may be chosen (0: barred), x the logits.  Slot j's expert on lane j, -1 for none.
// A round evaluates the experts within the margin of the largest fp32 choice, and
// none where they are alike (then the lowest index is right).
template <int V>
__device__ __noinline__ int choose_64(const float* x, uint32_t* key, const ScoreArgs& a, int E,
                                      int top_k, float top) {
  const int lane = threadIdx.x & 31;
  const double sum = a.sigmoid ? 1.0 : softmax_sum_64<V>(x, E, top);
  int mine = -1;
  for (int s = 0; s < top_k; ++s) {
    uint32_t best = 0;
    for (int i = 0; i < V; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(0xffffffffu, best);
    if (best == 0u) break;
    const float c = key_logit(best);
    // (of a NaN or an infinity only its equals, which go by index)
    const bool finite = c < __int_as_float(0x7f800000);
    const uint32_t from = finite ? logit_key(c - choice_margin(a.sigmoid, c)) : best;
    // the lowest candidate, and whether the others have its logit and bias
    uint32_t first = 0xffffffffu;
    for (int i = V - 1; i >= 0; --i)
      if (key[i] >= from && key[i] != 0u) first = uint32_t(i * 32 + lane);
    first = __reduce_min_sync(0xffffffffu, first);
    const float l0 = __shfl_sync(0xffffffffu, x[first >> 5], first & 31);
    const float b0 = a.bias ? __ldg(a.bias + first) : 0.0f;
    bool alike = true;
    for (int i = 0; i < V; ++i)
      if (key[i] >= from && key[i] != 0u &&
          (x[i] != l0 || (a.bias && __ldg(a.bias + i * 32 + lane) != b0)))
        alike = false;
    uint32_t pick = first;
    if (finite && !__all_sync(0xffffffffu, alike)) {
      double most = 0.0;
      uint32_t at = 0xffffffffu;
      for (int i = 0; i < V; ++i) {
        if (key[i] < from || key[i] == 0u) continue;
        const uint32_t e = uint32_t(i * 32 + lane);
        const double v =
            choice_64(x[i], a.bias ? __ldg(a.bias + e) : 0.0f, a.sigmoid, top, sum);
        if (at == 0xffffffffu || v > most) most = v, at = e;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const double v = shfl_xor_64(most, o);
        const uint32_t e = __shfl_xor_sync(0xffffffffu, at, o);
        if (e != 0xffffffffu && (at == 0xffffffffu || v > most || (v == most && e < at)))
          most = v, at = e;
      }
      pick = at;
    }
    if (lane == int(pick & 31)) key[pick >> 5] = 0u;
    if (lane == s) mine = int(pick);
  }
  return mine;
}

// The groups that stay, in fp64: bit g of the result.  A lane walks its own
// experts, a group at a time, and the warp joins them.
template <int V>
__device__ __noinline__ uint32_t groups_64(const float* x, const uint32_t* key,
                                           const ScoreArgs& a, int E, float top) {
  const int lane = threadIdx.x & 31;
  const double sum = a.sigmoid ? 1.0 : softmax_sum_64<V>(x, E, top);
  const int per = E / a.groups;
  // a token whose experts are all alike: groups by index, and by whether they have any
  bool alike = true;
  const float l0 = __shfl_sync(0xffffffffu, x[0], 0);
  const float b0 = a.bias ? __ldg(a.bias) : 0.0f;
  for (int i = 0; i < V; ++i) {
    const int e = i * 32 + lane;
    if (e < E && (x[i] != l0 || (a.bias && __ldg(a.bias + e) != b0))) alike = false;
  }
  alike = __all_sync(0xffffffffu, alike);
  double score = 0.0;       // of group `lane`
  bool any = false, nan = false;
  for (int g = 0; g < a.groups; ++g) {
    double m1 = 0.0, m2 = 0.0;
    int n = 0;              // of the two, how many there are
    bool bad = false;       // a NaN ranks its group above every number
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      if (key[i] == 0u || e < g * per || e >= (g + 1) * per) continue;
      const double v =
          alike ? 0.0 : choice_64(x[i], a.bias ? __ldg(a.bias + e) : 0.0f, a.sigmoid, top, sum);
      if (v != v) {
        bad = true;
      } else if (n == 0 || v > m1) {
        m2 = m1;
        m1 = v;
        n = n ? 2 : 1;
      } else if (n == 1 || v > m2) {
        m2 = v;
        n = 2;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double v1 = shfl_xor_64(m1, o), v2 = shfl_xor_64(m2, o);
      const int k = __shfl_xor_sync(0xffffffffu, n, o);
      if (k == 0) continue;
      if (n == 0) {
        m1 = v1, m2 = v2, n = k;
        continue;
      }
      // the two largest of m1 >= m2 and v1 >= v2
      const double hi = fmax(m1, v1), lo = fmin(m1, v1);
      double next = lo;
      if (v1 > m1) {
        if (k == 2 && v2 > next) next = v2;
      } else if (n == 2 && m2 > next) {
        next = m2;
      }
      m1 = hi, m2 = next, n = 2;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == g) {
      any = n > 0 || bad;
      nan = bad;
      score = a.group_top == 2 && n == 2 ? m1 + m2 : m1;
    }
  }
  int rank = 0;
  for (int g = 0; g < a.groups; ++g) {
    const double v = __shfl_sync(0xffffffffu, score, g);
    const bool has = __shfl_sync(0xffffffffu, any, g);
    const bool its = __shfl_sync(0xffffffffu, nan, g);
    const bool above = its || nan ? its && (!nan || g < lane)
                                  : v > score || (v == score && g < lane);
    if (has && (!any || above)) ++rank;
  }
  return __ballot_sync(0xffffffffu, lane < a.groups && any && rank < a.top_groups);
}

// The choice: lane j < top_k returns slot j in id (-1: none) and weight.  x: the
// logits, expert i * 32 + lane in x[i], -inf past E.  scratch: uint32[E] of this
// warp's, used where there are groups.
template <int V>
__device__ __forceinline__ void warp_choose(const float (&x)[V], const ScoreArgs& a, int E,
                                            int top_k, bool renormalize, uint32_t* scratch,
                                            int& id, float& weight) {
  const int lane = threadIdx.x & 31;
  const float ninf = __int_as_float(0xff800000);
  // softmax's statistics in fp32
  float top = 0.0f, sum = 1.0f;
  if (!a.sigmoid) {
    top = ninf;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, x[i]);
    top = warp_max(top);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * 32 + lane < E && x[i] != ninf) sum += expf(x[i] - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  const auto score_of = [&](float l) {
    return a.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-l)) : __fdividef(__expf(l - top), sum);
  };
  // keys of the choice, and of the groups' scores where those differ
  const bool by_logit = a.bias == nullptr;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 32 + lane;
    key[i] = 0u;
    if (e < E && x[i] != ninf) key[i] = logit_key(by_logit ? x[i] : score_of(x[i]) + __ldg(a.bias + e));
  }
  if (a.groups > 1) {
    bool again = false;     // decide in fp64
    const bool exact = by_logit && a.group_top == 1;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      if (e < E)
        scratch[e] = by_logit && !exact && key[i] != 0u ? logit_key(score_of(x[i])) : key[i];
    }
    __syncwarp();
    // a group per 2^n lanes, which share out its experts
    int lanes = 32;
    while (lanes * a.groups > 32) lanes >>= 1;
    const int per = E / a.groups, g = lane / lanes;
    uint32_t k1 = 0, k2 = 0;
    if (g < a.groups)
      for (int j = lane % lanes; j < per; j += lanes) {
        const uint32_t k = scratch[g * per + j];
        k2 = max(k2, min(k1, k));
        k1 = max(k1, k);
      }
    for (int o = 1; o < lanes; o <<= 1) {
      const uint32_t v1 = __shfl_xor_sync(0xffffffffu, k1, o);
      const uint32_t v2 = __shfl_xor_sync(0xffffffffu, k2, o);
      k2 = max(max(k2, v2), min(k1, v1));
      k1 = max(k1, v1);
    }
    uint32_t score = k1;
    if (a.group_top == 2 && k2 != 0u) {
      score = logit_key(key_logit(k1) + key_logit(k2));
      if (score == 0u) score = 1u;      // (-inf, of choices that are not barred)
    }
    int rank = 0;
    for (int h = 0; h < a.groups; ++h) {
      const uint32_t v = __shfl_sync(0xffffffffu, score, h * lanes);
      rank += v > score || (v == score && h < g);
    }
    const bool stays = g < a.groups && score != 0u && rank < a.top_groups;
    uint32_t kept = __ballot_sync(0xffffffffu, stays && lane % lanes == 0);
    if (!exact) {
      const uint32_t in = __reduce_min_sync(0xffffffffu, stays ? score : 0xffffffffu);
      const uint32_t out =
          __reduce_max_sync(0xffffffffu, g < a.groups && !stays ? score : 0u);
      if (out != 0u && in != 0xffffffffu) {
        const float vi = key_logit(in), vo = key_logit(out);
        again = vi - vo < 2.0f * choice_margin(a.sigmoid, vi) || in == out;
      }
    }
    if (again) {
      float xs[V];          // (copies, so that x and key stay in registers)
      uint32_t keys[V];
#pragma unroll
      for (int i = 0; i < V; ++i) xs[i] = x[i], keys[i] = key[i];
      const uint32_t by_group = groups_64<V>(xs, keys, a, E, top);
      kept = 0u;
      for (int h = 0; h < a.groups; ++h) kept |= (by_group >> h & 1u) << (h * lanes);
    }
    // the experts of the other groups are barred
    if (g < a.groups && !(kept >> (g * lanes) & 1u))
      for (int j = lane % lanes; j < per; j += lanes) scratch[g * per + j] = 0u;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 32 + lane;
      if (e < E && scratch[e] == 0u) key[i] = 0u;
    }
  }
  // the slots, and with a bias the expert that comes next, for its margin
  const int rounds = by_logit ? top_k : top_k + 1;
  uint32_t beyond = 0u;
  uint32_t left[V];
#pragma unroll
  for (int i = 0; i < V; ++i) left[i] = key[i];
  id = -1;
  uint32_t mine = 0u;
  for (int s = 0; s < rounds; ++s) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) best = max(best, left[i]);
    const uint32_t all = __reduce_max_sync(0xffffffffu, best);
    if (all == 0u) break;
    uint32_t e = 0xffffffffu;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (left[i] == all) e = uint32_t(i * 32 + lane);
    const uint32_t pick = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (uint32_t(i * 32 + lane) == pick) left[i] = 0u;
    if (lane == s) id = int(pick), mine = all;
    beyond = all;
  }
  // this slot's logit
  const auto logit_of = [&](int e) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float w = __shfl_sync(0xffffffffu, x[i], e & 31);
      if (i == e >> 5) v = w;
    }
    return v;
  };
  float l = logit_of(max(id, 0));
  if (!by_logit) {
    const float b = id >= 0 ? __ldg(a.bias + id) : 0.0f;
    uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
    const float next_l = __shfl_down_sync(0xffffffffu, l, 1);
    const float next_b = __shfl_down_sync(0xffffffffu, b, 1);
    // (of the last slot and the expert beyond not: another may be as near behind it)
    const bool alike = lane + 1 < top_k && l == next_l && b == next_b;
    if (lane == 31) next = top_k == 32 && E > 32 ? beyond : 0u;
    bool near = false;
    if (lane < top_k && mine != 0u && next != 0u && !alike) {
      const float c = key_logit(mine);
      near = mine == next || c - key_logit(next) < choice_margin(a.sigmoid, c);
    }
    if (__any_sync(0xffffffffu, near)) {
      float xs[V];
      uint32_t keys[V];
#pragma unroll
      for (int i = 0; i < V; ++i) xs[i] = x[i], keys[i] = key[i];
      id = choose_64<V>(xs, keys, a, E, top_k, top);
      l = logit_of(max(id, 0));
    }
  }
  if (lane >= top_k) id = -1;
  // the weights, in fp32.  Chosen scores may all be far below 1, so sigmoids to be
  // renormalised share a factor that makes the largest about 1.
  float s = 0.0f;
  if (id >= 0) {
    if (a.sigmoid) {
      s = 1.0f / (1.0f + expf(-l));
    } else {
      s = expf(l - top) / sum;
    }
  }
  if (renormalize) {
    if (a.sigmoid) {
      // e^(l - m) / (1 + e^l) with m the largest chosen logit, where that is negative
      const float m = fminf(warp_max(id >= 0 ? l : ninf), 0.0f);
      if (id >= 0 && l < 0.0f) s = expf(l - m) / (1.0f + expf(l));
      else if (id >= 0) s = 1.0f / (1.0f + expf(-l));
    } else {
      // softmax over the chosen, whatever share of the whole they have (a NaN or +inf
      // anywhere enters every score)
      const float m = warp_max(id >= 0 ? l : ninf);
      s = id >= 0 ? (sum == sum ? expf(l - m) : sum) : 0.0f;
    }
    float all = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    s = id >= 0 ? s / all : 0.0f;
  }
  weight = id >= 0 ? a.scale * s : 0.0f;
}

}  // namespace fo
