// A whole expert layer for a few tokens:
//   y[t] = sum_s w_s W2[e_s] (act(G x_t) * (U x_t)),  ids, w = top-k softmax
// of x . router^T.
//
// The plain first form, one warp per value: the router with a CTA per token,
// the hidden values with a warp per (token, slot, hidden row), the outputs
// with a warp per (token, output row).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "moe_common.cuh"
#include "mx_common.cuh"

namespace fo {

namespace {

struct FewArgs {
  fo_moe_few_desc d;
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* router;
  const void *w1, *w2;
  const uint8_t *s1, *s2;
  uint16_t* y;
  int64_t y_stride;
  int32_t* ids;
  float* weights;
  float* h;
};

__device__ __forceinline__ float bf16_at(const uint16_t* p, int64_t i) {
  return __uint_as_float(uint32_t(p[i]) << 16);
}

// Element (row, k) of a 4-bit matrix whose first row is row 0 of `codes`.
__device__ float mx_at(const uint8_t* codes, const uint8_t* scales, int64_t row, int64_t k,
                       int64_t k_blocks) {
  const uint32_t byte = codes[row * k_blocks * 64 + k / 2];
  uint32_t h[4];
  mx_decode8((k & 1) ? byte >> 4 : byte & 15, h);
  const float v = __half2float(__low2half(*reinterpret_cast<const __half2*>(&h[0])));
  return v * mx_scale_value(scales[((row / 128) * k_blocks + k / 128) * 512 +
                                   mx_scale_row(int(row % 128)) + (k % 128) / 32]);
}

__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int V>
__global__ void few_router_kernel(const FewArgs a) {
  __shared__ float logits[kRouteExperts];
  const int t = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int H = a.d.hidden, E = a.d.experts;
  for (int e = warp; e < E; e += blockDim.x / 32) {
    float s = 0;
    for (int k = lane; k < H; k += 32)
      s += bf16_at(a.x, t * a.x_stride + k) * bf16_at(a.router, int64_t(e) * H + k);
    s = warp_sum(s);
    if (lane == 0) logits[e] = s;
  }
  __syncthreads();
  if (warp) return;
  float x[V];
  for (int i = 0; i < V; ++i)
    x[i] = i * 32 + lane < E ? logits[i * 32 + lane] : __int_as_float(0xff800000);
  int id;
  float w;
  warp_top_k<V>(x, E, a.d.top_k, a.d.renormalize != 0, id, w);
  if (lane < a.d.top_k) {
    a.ids[t * a.d.top_k + lane] = id;
    a.weights[t * a.d.top_k + lane] = w;
  }
}

__global__ void few_hidden_kernel(const FewArgs a) {
  const int H = a.d.hidden, I = a.d.inter, K = a.d.top_k, lane = threadIdx.x % 32;
  const int64_t job = int64_t(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  const int64_t p = job / I, i = job % I;
  if (p >= int64_t(a.d.tokens) * K) return;
  const int e = a.ids[p];
  if (e < 0) return;
  const int64_t kb = mx_up(H, 128) / 128, rows = mx_up(2 * int64_t(I), 128);
  float g = 0, u = 0;
  for (int k = lane; k < H; k += 32) {
    const float x = bf16_at(a.x, (p / K) * a.x_stride + k);
    if (a.d.weights == FO_TYPE_BF16) {
      const uint16_t* w = static_cast<const uint16_t*>(a.w1) + int64_t(e) * 2 * I * H;
      g += x * bf16_at(w, i * H + k);
      u += x * bf16_at(w, (I + i) * H + k);
    } else {
      const uint8_t* w = static_cast<const uint8_t*>(a.w1);
      g += x * mx_at(w, a.s1, e * rows + i, k, kb);
      u += x * mx_at(w, a.s1, e * rows + I + i, k, kb);
    }
  }
  g = warp_sum(g);
  u = warp_sum(u);
  if (lane == 0) a.h[p * I + i] = (a.d.act == FO_ACT_NONE   ? g
                                   : a.d.act == FO_ACT_RELU ? (g > 0 ? g : 0.0f)
                                                            : g / (1.0f + expf(-g))) * u;
}

__global__ void few_output_kernel(const FewArgs a) {
  const int H = a.d.hidden, I = a.d.inter, K = a.d.top_k, lane = threadIdx.x % 32;
  const int64_t job = int64_t(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  const int64_t t = job / H, r = job % H;
  if (t >= a.d.tokens) return;
  const int64_t kb = mx_up(I, 128) / 128, rows = mx_up(H, 128);
  float y = 0;
  for (int s = 0; s < K; ++s) {
    const int e = a.ids[t * K + s];
    if (e < 0) continue;
    float v = 0;
    for (int k = lane; k < I; k += 32) {
      const float h = a.h[(t * K + s) * I + k];
      if (a.d.weights == FO_TYPE_BF16)
        v += h * bf16_at(static_cast<const uint16_t*>(a.w2), (int64_t(e) * H + r) * I + k);
      else
        v += h * mx_at(static_cast<const uint8_t*>(a.w2), a.s2, e * rows + r, k, kb);
    }
    y += a.weights[t * K + s] * warp_sum(v);
  }
  if (lane == 0)
    reinterpret_cast<__nv_bfloat16*>(a.y)[t * a.y_stride + r] = __float2bfloat16_rn(y);
}

}  // namespace

int64_t few_workspace_bytes(const fo_moe_few_desc& d) {
  const int64_t pairs = int64_t(d.tokens) * d.top_k;
  return 256 + mx_up(8 * pairs, 256) + 4 * pairs * d.inter;
}

fo_status launch_moe_few(const fo_moe_few_desc& d, const void* x, int64_t x_stride,
                         const void* router, const void* W1, const void* S1, const void* W2,
                         const void* S2, void* y, int64_t y_stride, void* workspace,
                         int32_t*, void* stream) {
  if (d.tokens == 0) return FO_OK;
  const int64_t pairs = int64_t(d.tokens) * d.top_k;
  uint8_t* ws = static_cast<uint8_t*>(workspace) + 256;
  FewArgs a{d, static_cast<const uint16_t*>(x), x_stride, static_cast<const uint16_t*>(router),
            W1, W2, static_cast<const uint8_t*>(S1), static_cast<const uint8_t*>(S2),
            static_cast<uint16_t*>(y), y_stride, reinterpret_cast<int32_t*>(ws),
            reinterpret_cast<float*>(ws + 4 * pairs),
            reinterpret_cast<float*>(ws + mx_up(8 * pairs, 256))};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d.experts <= 256)
    few_router_kernel<8><<<d.tokens, 256, 0, st>>>(a);
  else
    few_router_kernel<32><<<d.tokens, 256, 0, st>>>(a);
  few_hidden_kernel<<<unsigned((pairs * d.inter + 7) / 8), 256, 0, st>>>(a);
  few_output_kernel<<<unsigned((int64_t(d.tokens) * d.hidden + 7) / 8), 256, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace fo
