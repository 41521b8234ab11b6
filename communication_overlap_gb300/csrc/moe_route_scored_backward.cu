// Gradient of the balanced router's weights (moe_scores.cuh).  For a token with
// w = scale s / sum (renormalised) or scale s, and g the weights' gradient, dot = sum
// of w g over its slots, at a chosen expert:
//   sigmoid, renormalised: w (1 - s) (g - dot / scale)    since ds / dl = s (1 - s)
//   sigmoid:               w (1 - s) g
//   softmax, renormalised: w (g - dot / scale)
//   softmax:               w g - p dot, and -p dot at every other expert
// elsewhere zero.  The bias decides the choice only and has no gradient.
//
// A warp per token writes the row (zeros, in 16 bytes per lane, while the slots are on
// their way; or -p dot), then its slots.  16384 x 256 in fp32: 4.9 us within a graph
// (5.7 with a lane's element per store), 11.4 where softmax's sum is formed again.
#include <cuda_runtime.h>

#include "moe_common.cuh"

namespace fo {

namespace {

struct BackArgs {
  const void* logits;
  int64_t stride;
  int32_t bf16, experts, top_k, renormalize, sigmoid;
  float scale;
  int64_t tokens;
  const int32_t* ids;
  const float* weights;
  const float* dweights;
  void* dlogits;
  int64_t dstride;
};

__device__ __forceinline__ float logit_at(const BackArgs& a, int64_t i) {
  return a.bf16 ? __uint_as_float(uint32_t(static_cast<const uint16_t*>(a.logits)[i]) << 16)
                : static_cast<const float*>(a.logits)[i];
}

__device__ __forceinline__ void put(const BackArgs& a, int64_t i, float v) {
  if (a.bf16)
    static_cast<__nv_bfloat16*>(a.dlogits)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(a.dlogits)[i] = v;
}

// A row of zeros, by a warp.
__device__ __forceinline__ void put_zeros(const BackArgs& a, int64_t at) {
  const int lane = threadIdx.x & 31, size = a.bf16 ? 2 : 4;
  char* p = static_cast<char*>(a.dlogits) + at * size;
  int bytes = 0;                // that were written in wide stores
  if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    bytes = a.experts * size & ~15;
    for (int i = lane * 16; i < bytes; i += 512)
      *reinterpret_cast<int4*>(p + i) = make_int4(0, 0, 0, 0);
  }
  for (int e = bytes / size + lane; e < a.experts; e += 32) put(a, at + e, 0.0f);
}

__global__ void __launch_bounds__(256) scored_backward_kernel(const BackArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t t = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (t >= a.tokens) return;
  const int E = a.experts, K = a.top_k;
  const bool zeros = a.sigmoid || a.renormalize;      // but at the chosen
  const int64_t to = t * a.dstride, from = t * a.stride;
  int id = -1;
  float w = 0.0f, g = 0.0f;
  if (lane < K) {
    id = a.ids[t * K + lane];
    w = a.weights[t * K + lane];
    g = a.dweights[t * K + lane];
  }
  if (zeros) put_zeros(a, to);
  if (id < 0 || id >= E) id = -1, w = g = 0.0f;
  float dot = w * g;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  float d = 0.0f;
  if (a.sigmoid) {
    // 1 - s = 1 / (1 + e^l)
    if (id >= 0)
      d = w * (a.renormalize ? g - dot / a.scale : g) / (1.0f + expf(logit_at(a, from + id)));
  } else if (a.renormalize) {
    d = w * (g - dot / a.scale);
  }
  if (!zeros) {
    const float ninf = __int_as_float(0xff800000);
    float top = ninf;
    for (int e = lane; e < E; e += 32) top = fmaxf(top, logit_at(a, from + e));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool none = top == ninf;      // every expert barred
    float sum = 0.0f;
    for (int e = lane; e < E; e += 32) sum += none ? 0.0f : expf(logit_at(a, from + e) - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    for (int e = lane; e < E; e += 32)
      put(a, to + e, none ? 0.0f : -(expf(logit_at(a, from + e) - top) / sum) * dot);
    if (id >= 0) d = w * g - expf(logit_at(a, from + id) - top) / sum * dot;
  }
  __syncwarp();       // the slots' stores come after the row's
  if (id >= 0) put(a, to + id, d);
}

}  // namespace

fo_status launch_moe_route_scored_backward(const fo_route_desc& d, const void* logits,
                                           fo_type type, int64_t tokens, int64_t row_stride,
                                           const int32_t* ids, const float* weights,
                                           const float* dweights, void* dlogits,
                                           int64_t dlogits_stride, void* stream) {
  const BackArgs a{logits, row_stride, type == FO_TYPE_BF16, d.experts, d.top_k,
                   d.renormalize != 0, d.score == FO_SCORE_SIGMOID, d.scale, tokens, ids,
                   weights, dweights, dlogits, dlogits_stride};
  scored_backward_kernel<<<unsigned((tokens + 7) / 8), 256, 0,
                           static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace fo
