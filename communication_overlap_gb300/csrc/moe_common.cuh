// Device helpers of the expert layer's kernels: the top-k choice of one
// token by one warp, and the barrier of a cooperative grid.
#pragma once

#include <cstdint>

#include "device_common.cuh"
#include "moe_internal.h"

namespace fo {

constexpr uint64_t kGridWaitNs = 2000000000ull;

// Order-preserving key of a logit: larger logit, larger key; +0 and -0 equal;
// a NaN above everything; -inf 0 (barred: every other key is larger).
__device__ __forceinline__ uint32_t logit_key(float x) {
  if (x != x) return 0xffffffffu;
  if (x == __int_as_float(0xff800000)) return 0u;
  const uint32_t b = __float_as_uint(x + 0.0f);   // -0 becomes +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The logit of a key (a NaN for a NaN's).
__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// The top_k largest of a token's E logits, held V per lane (expert e = i * 32
// + lane in x[i]; -inf past E), and their weights.  Lane j < top_k returns
// slot j in id and weight.
//
// A round takes the largest key over lanes with one integer reduction and,
// among the lanes that hold it, the lowest expert with a second, so ties go to
// the lowest index.
template <int V>
__device__ __forceinline__ void warp_top_k(const float (&x)[V], int E, int top_k,
                                           bool renormalize, int& id, float& weight) {
  const int lane = threadIdx.x & 31;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = i * 32 + lane < E ? logit_key(x[i]) : 0u;
  id = -1;
  float mine = 0.0f;      // this slot's logit
  bool bad = false;       // the row holds a NaN or +inf
  float top = 0.0f;
  for (int s = 0; s < top_k; ++s) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) best = max(best, key[i]);
    const uint32_t all = __reduce_max_sync(0xffffffffu, best);
    if (all == 0u) break;   // every expert left is barred
    uint32_t e = 0xffffffffu;
    float l = 0.0f;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (key[i] == all) e = uint32_t(i * 32 + lane), l = x[i];
    const uint32_t pick = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (uint32_t(i * 32 + lane) == pick) key[i] = 0u;
    // the logit from its lane, or with many per lane back from the key (65536 x
    // 256 tokens, top 8: 92 us and 101; 16384 x 1024, top 32: 223 and 183)
    l = V <= 8 ? __shfl_sync(0xffffffffu, l, pick & 31) : key_logit(all);
    if (s == 0) {
      top = l;
      bad = !(l < __int_as_float(0x7f800000));   // +inf or NaN
    }
    if (lane == s) id = int(pick), mine = l;
  }
  // softmax statistics in fp32; the butterfly adds in the same order on every
  // lane and in every run
  float e = id >= 0 ? expf(mine - top) : 0.0f;
  float sum = 0.0f;
  if (renormalize) {
    sum = e;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * 32 + lane < E) sum += expf(x[i] - top);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  weight = id >= 0 ? e / sum : 0.0f;
  if (bad && id >= 0) weight = __int_as_float(0x7fffffff);
}

// Barrier over all CTAs of a cooperative launch, for one thread per CTA:
// count rises to the grid's size.  `count` starts at 0 and a later
// grid_barrier_leave resets it; several barriers use several words.  Bounded:
// false when the wait ran out (recorded in *status).
__device__ __forceinline__ bool grid_barrier(uint32_t* count, uint32_t target, int32_t* status) {
  uint32_t old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(count) : "memory");
  if (old + 1 == target) return true;
  uint64_t t0 = 0;
  for (uint32_t i = 1; ld_acquire_gpu(count) < target; ++i) {
    if (i % 64) continue;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kGridWaitNs) {
      atomicCAS(status, 0, int32_t(FO_ERR_TIMEOUT));
      return false;
    }
  }
  return true;
}

// Every CTA calls this once when it is past all barriers; the last one zeroes
// the `n` words at `count` and the leave counter for the next launch.
__device__ __forceinline__ void grid_barrier_leave(uint32_t* leave, uint32_t* count, int n,
                                                   uint32_t ctas) {
  uint32_t old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(leave) : "memory");
  if (old + 1 == ctas) {
    for (int i = 0; i < n; ++i) st_release_gpu(count + i, 0u);
    st_release_gpu(leave, 0u);
  }
}

}  // namespace fo
