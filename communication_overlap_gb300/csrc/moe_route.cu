// The router: top-k choice, softmax weights, row tables, and the gradient.
//
// For a token's logits l: p_e = exp(l_e - max l) / sum_j exp(l_j - max l); the
// chosen experts are the top_k largest, and the row tables are a stable
// counting sort of the (token, slot) pairs by expert:
//   row(t, s) = first[e] + |{(t', s') before (t, s): id(t', s') = e}|.
//
// One cooperative kernel.  CTA c owns a contiguous chunk of tokens, a warp
// one token at a time:
//   1. choose, write ids and weights, keep the chunk's ids in shared memory,
//      count them per expert, and mark this CTA's share of the row tables empty;
//   2. grid barrier, with the counts of every chunk in global memory;
//   3. sum the counts of the earlier chunks (this chunk's start per expert)
//      and of all chunks (the experts' ranges), and place the chunk's pairs:
//      a warp's sub-chunk starts where the earlier warps' counts end, and
//      inside it 32 pairs at a time rank themselves with a warp match.
// Counts are integers, so the order of the additions does not matter, and the
// tables are the same in every run.  The work is a few bytes per logit; what
// bounds it is latency (launch, barrier, the chain of rounds), so there is one
// launch, and up to 16 tokens run in one CTA without the barrier.
//
// Measured: 6 us for 1 token of 64 logits, top 8; 14.5 us for 16384 tokens of 8,
// top 2; 27 us for 16384 of 128, top 8 (its bytes take 2 us at HBM's rate), 92 us
// for 65536 of 256: there the rounds bind, some 25 instructions each per token.
// Two CTAs per SM, or a vote instead of the second reduction of a round, are no
// faster.  The gradient: 10 us for 16384 of 128.
#include <cuda_runtime.h>

#include <mutex>

#include "moe_common.cuh"

namespace fo {

namespace {

constexpr int kRouteWarps = 16;
constexpr int kRouteThreads = kRouteWarps * 32;
constexpr int kRouteSmemLimit = 200 * 1024;   // that a launch asks for (8 KB more are static)

__device__ __forceinline__ float load_logit(const void* p, int64_t i, bool bf16) {
  return bf16 ? __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i]) << 16)
              : static_cast<const float*>(p)[i];
}

struct RouteKernelArgs {
  const void* logits;
  int64_t stride;
  int32_t bf16, tokens, experts, top_k, renormalize;
  int64_t capacity, table_rows;
  int32_t* ids;
  float* weights;
  int32_t* row_token;
  int32_t* row_slot;
  int32_t* token_row;
  int32_t* expert_first;
  int32_t* expert_rows;
  uint32_t* barrier;   // [0] count, [1] leave
  int32_t* counts;     // [grid][experts] pairs of each chunk per expert
  int32_t* status;
  int32_t chunk;       // tokens per CTA
};

// Shared memory: ids of the chunk where they fit (1056 tokens of top 32 over 1024
// experts do, 160512 on 152 SMs; a larger chunk reads them back from the output),
// per-warp counts (then starts) per expert, the chunk's start per expert.  (Ids last:
// 28.8 us instead of 26.7 for 16384 tokens of 128 experts.)
__host__ __device__ inline int64_t route_smem(int64_t kept, int experts) {
  return 4 * (kept + int64_t(kRouteWarps + 1) * experts);
}

// KEPT: the chunk's ids stay in shared memory.  (Decided at run time, 100000 tokens
// of 128 experts take 104 us, not 100.)
template <int V, bool KEPT>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteKernelArgs a) {
  extern __shared__ int32_t sm[];
  const int E = a.experts, K = a.top_k;
  int32_t* cnt = KEPT ? sm + int64_t(a.chunk) * K : sm;    // [kRouteWarps][E]
  int32_t* start = cnt + kRouteWarps * E;              // [E]
  __shared__ int32_t ok_s;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t t0 = int64_t(blockIdx.x) * a.chunk;
  const int n = int(min(int64_t(a.chunk), int64_t(a.tokens) - t0));   // > 0 by the grid's size
  const int pairs = n * K;
  int32_t* ids = KEPT ? sm : a.ids + t0 * K;           // [chunk * K]
  // a warp's sub-chunk of pairs, whole groups of 32
  const int per_warp = ((pairs + kRouteWarps * 32 - 1) / (kRouteWarps * 32)) * 32;

  for (int i = threadIdx.x; i < kRouteWarps * E; i += kRouteThreads) cnt[i] = 0;
  // this CTA's share of the row tables starts empty
  {
    const int64_t share = (a.table_rows + gridDim.x - 1) / gridDim.x;
    const int64_t lo = share * blockIdx.x, hi = min(lo + share, a.table_rows);
    for (int64_t i = lo + threadIdx.x; i < hi; i += kRouteThreads) {
      a.row_token[i] = -1;
      a.row_slot[i] = 0;
    }
  }
  // a token's logits are on their way while the one before it is chosen for,
  // where a warp has registers for both
  auto load = [&](int t, float (&x)[V]) {
    const int64_t at = (t0 + t) * a.stride;
#pragma unroll
    for (int i = 0; i < V; ++i)
      x[i] = t < n && i * 32 + lane < E
                 ? load_logit(a.logits, at + i * 32 + lane, a.bf16 != 0)
                 : __int_as_float(0xff800000);
  };
  constexpr bool kAhead = V <= 8;
  float ahead[V];
  if (kAhead) load(warp, ahead);
  for (int t = warp; t < n; t += kRouteWarps) {
    float x[V];
    if (kAhead) {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = ahead[i];
      load(t + kRouteWarps, ahead);
    } else {
      load(t, x);
    }
    int id;
    float w;
    warp_top_k<V>(x, E, K, a.renormalize != 0, id, w);
    if (lane < K) {
      ids[t * K + lane] = id;
      a.ids[(t0 + t) * K + lane] = id;
      a.weights[(t0 + t) * K + lane] = w;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += kRouteThreads) {
    const int e = ids[i];
    if (e >= 0) atomicAdd(&cnt[(i / per_warp) * E + e], 1);
  }
  __syncthreads();
  const bool alone = gridDim.x == 1;
  // per expert: the chunk's total, and each warp's start inside the chunk
  for (int e = threadIdx.x; e < E; e += kRouteThreads) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kRouteWarps; ++w) {
      const int c = cnt[w * E + e];
      cnt[w * E + e] = sum;
      sum += c;
    }
    start[e] = sum;
    if (!alone) __stcg(a.counts + int64_t(blockIdx.x) * E + e, sum);
  }
  if (!alone) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) ok_s = grid_barrier(a.barrier, gridDim.x, a.status);
    __syncthreads();
    if (threadIdx.x == 0) grid_barrier_leave(a.barrier + 1, a.barrier, 1, gridDim.x);
    if (!ok_s) return;
  }
  __syncthreads();
  // earlier chunks' pairs per expert and the total, then the experts' ranges
  __shared__ int32_t total[kRouteExperts];
  if (alone) {
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
      total[e] = start[e];
      start[e] = 0;
    }
  } else {
    // several threads per expert share out the chunks (with one each 16384 tokens
    // over 8 experts took 17.4 us, not 14.5)
    for (int e = threadIdx.x; e < E; e += kRouteThreads) total[e] = start[e] = 0;
    __syncthreads();
    const int parts = max(kRouteThreads / E, 1);
    for (int i = threadIdx.x; i < E * parts; i += kRouteThreads) {
      const int e = i % E;
      int before = 0, all = 0;
#pragma unroll 8
      for (int c = i / E; c < int(gridDim.x); c += parts) {
        const int v = __ldcg(a.counts + int64_t(c) * E + e);
        before += c < int(blockIdx.x) ? v : 0;
        all += v;
      }
      atomicAdd(&total[e], all);        // (integers: in any order)
      if (before) atomicAdd(&start[e], before);
    }
  }
  __syncthreads();
  __shared__ int32_t first[kRouteExperts];
  if (warp == 0) {
    int64_t at = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int rows = e < E ? total[e] : 0;
      int span = (rows + 127) & ~127;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, span, o);
        if (lane >= o) span += v;
      }
      const int sum = __shfl_sync(0xffffffffu, span, 31);
      if (e < E) {
        const int f = a.capacity ? int(int64_t(e) * a.capacity)
                                 : int(at) + span - ((rows + 127) & ~127);
        first[e] = f;
        if (blockIdx.x == 0) {
          a.expert_first[e] = f;
          a.expert_rows[e] = a.capacity ? int(min(int64_t(rows), a.capacity)) : rows;
        }
      }
      at += sum;
    }
  }
  __syncthreads();
  // place the pairs: rank inside the warp's sub-chunk by a match of 32
  int32_t* run = cnt + warp * E;
  const int lo = warp * per_warp, hi = min(lo + per_warp, pairs);
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const int e = i < hi ? ids[i] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int row = -1;
    if (e >= 0) {
      const int pos = start[e] + run[e] + rank;
      if (a.capacity == 0 || pos < a.capacity) row = first[e] + pos;
    }
    __syncwarp();
    if (e >= 0 && rank == 0) run[e] += __popc(same);
    __syncwarp();
    if (i < hi) {
      const int64_t t = t0 + i / K;
      a.token_row[t0 * K + i] = row;
      if (row >= 0) {
        a.row_token[row] = int32_t(t);
        a.row_slot[row] = i % K;
      }
    }
  }
}

struct RouteBackArgs {
  const void* logits;
  int64_t stride;
  int32_t bf16, experts, top_k, renormalize;
  int64_t tokens;
  const int32_t* ids;
  const float* weights;
  const float* dweights;
  void* dlogits;
  int64_t dstride;
};

// A warp per token; the sums in fp32, one rounding to the logits' type.
template <int V>
__global__ void __launch_bounds__(256) route_backward_kernel(const RouteBackArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t t = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (t >= a.tokens) return;
  const int E = a.experts, K = a.top_k;
  int id = -1;
  float w = 0.0f, g = 0.0f;
  if (lane < K) {
    id = a.ids[t * K + lane];
    if (id >= 0 && id < E) {
      w = a.weights[t * K + lane];
      g = a.dweights[t * K + lane];
    } else {
      id = -1;
    }
  }
  float dot = w * g;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  float d[V];
  if (a.renormalize) {
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.0f;
  } else {
    float x[V], top = __int_as_float(0xff800000);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = i * 32 + lane < E ? load_logit(a.logits, t * a.stride + i * 32 + lane, a.bf16 != 0)
                               : __int_as_float(0xff800000);
      top = fmaxf(top, x[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = 0.0f;
    const bool none = top == __int_as_float(0xff800000);   // every expert barred
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = none ? 0.0f : expf(x[i] - top);
      sum += x[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = none ? 0.0f : -(x[i] / sum) * dot;
  }
  // the chosen experts' own term, slot by slot (distinct experts)
  for (int s = 0; s < K; ++s) {
    const int e = __shfl_sync(0xffffffffu, id, s);
    const float ws = __shfl_sync(0xffffffffu, w, s), gs = __shfl_sync(0xffffffffu, g, s);
    if (e < 0) continue;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * 32 + lane == e) d[i] = ws * (gs - dot);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 32 + lane;
    if (e >= E) continue;
    if (a.bf16)
      static_cast<__nv_bfloat16*>(a.dlogits)[t * a.dstride + e] = __float2bfloat16_rn(d[i]);
    else
      static_cast<float*>(a.dlogits)[t * a.dstride + e] = d[i];
  }
}

// Tokens per CTA: at least a warp's worth each, and no more CTAs than SMs so
// that the barrier's grid is resident at once.
int64_t route_chunk(int64_t tokens, int sms) {
  int64_t chunk = (tokens + sms - 1) / sms;
  return chunk < kRouteWarps ? kRouteWarps : chunk;
}

fo_status sm_count(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FO_ERR_CUDA;
  return FO_OK;
}

template <int V, bool KEPT>
fo_status launch_as(const RouteKernelArgs& a, int grid, int smem, cudaStream_t st) {
  // the limit once, not each launch's size: that would be lowered between another
  // thread's setting and its launch, and 48 KB bound the static part's sum with it
  static std::once_flag once[64];
  static cudaError_t err[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FO_ERR_CUDA;
  const int slot = dev < 64 ? dev : 63;
  std::call_once(once[slot], [&] {
    err[slot] =
        cudaFuncSetAttribute(route_kernel<V, KEPT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kRouteSmemLimit);
  });
  if (err[slot] != cudaSuccess) return FO_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kRouteThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = grid > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, route_kernel<V, KEPT>, a) != cudaSuccess) {
    cudaGetLastError();
    return FO_ERR_CUDA;
  }
  return FO_OK;
}

template <int V>
fo_status launch_v(const RouteKernelArgs& a, int grid, cudaStream_t st) {
  const int64_t kept = route_smem(int64_t(a.chunk) * a.top_k, a.experts);
  if (kept <= kRouteSmemLimit) return launch_as<V, true>(a, grid, int(kept), st);
  return launch_as<V, false>(a, grid, int(route_smem(0, a.experts)), st);
}

}  // namespace

// Bytes of the workspace: the barrier's words, then counts for as many chunks
// as any device of this kind runs CTAs.
constexpr int64_t kRouteMaxCtas = 1024;
int64_t route_workspace_bytes(int experts) { return 256 + kRouteMaxCtas * 4 * int64_t(experts); }

fo_status launch_moe_route(const void* logits, fo_type type, int64_t tokens, int32_t experts,
                           int64_t row_stride, int32_t top_k, bool renormalize,
                           int64_t capacity, int64_t table_rows, int32_t* ids, float* weights,
                           int32_t* row_token, int32_t* row_slot, int32_t* token_row,
                           int32_t* expert_first, int32_t* expert_rows, void* workspace,
                           int32_t* dev_status, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int sms = 0;
  const fo_status q = sm_count(&sms);
  if (q != FO_OK) return q;
  if (sms > kRouteMaxCtas) sms = int(kRouteMaxCtas);
  RouteKernelArgs a{};
  a.logits = logits;
  a.stride = row_stride;
  a.bf16 = type == FO_TYPE_BF16;
  a.tokens = int32_t(tokens);
  a.experts = experts;
  a.top_k = top_k;
  a.renormalize = renormalize;
  a.capacity = capacity;
  a.table_rows = table_rows;
  a.ids = ids;
  a.weights = weights;
  a.row_token = row_token;
  a.row_slot = row_slot;
  a.token_row = token_row;
  a.expert_first = expert_first;
  a.expert_rows = expert_rows;
  a.barrier = static_cast<uint32_t*>(workspace);
  a.counts = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + 256);
  a.status = dev_status;
  const int64_t chunk = route_chunk(tokens, sms);
  a.chunk = int32_t(chunk);
  const int grid = tokens == 0 ? 1 : int((tokens + chunk - 1) / chunk);
  const int v = (experts + 31) / 32;
  if (v <= 1) return launch_v<1>(a, grid, st);
  if (v <= 2) return launch_v<2>(a, grid, st);
  if (v <= 4) return launch_v<4>(a, grid, st);
  if (v <= 8) return launch_v<8>(a, grid, st);
  if (v <= 16) return launch_v<16>(a, grid, st);
  return launch_v<32>(a, grid, st);
}

fo_status launch_moe_route_backward(const void* logits, fo_type type, int64_t tokens,
                                    int32_t experts, int64_t row_stride, int32_t top_k,
                                    bool renormalize, const int32_t* ids, const float* weights,
                                    const float* dweights, void* dlogits,
                                    int64_t dlogits_stride, void* stream) {
  if (tokens == 0) return FO_OK;
  RouteBackArgs a{logits, row_stride, type == FO_TYPE_BF16, experts, top_k, renormalize, tokens,
                  ids, weights, dweights, dlogits, dlogits_stride};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = unsigned((tokens + 7) / 8);
  const int v = (experts + 31) / 32;
  if (v <= 1)
    route_backward_kernel<1><<<grid, 256, 0, st>>>(a);
  else if (v <= 2)
    route_backward_kernel<2><<<grid, 256, 0, st>>>(a);
  else if (v <= 4)
    route_backward_kernel<4><<<grid, 256, 0, st>>>(a);
  else if (v <= 8)
    route_backward_kernel<8><<<grid, 256, 0, st>>>(a);
  else if (v <= 16)
    route_backward_kernel<16><<<grid, 256, 0, st>>>(a);
  else
    route_backward_kernel<32><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA;
}

}  // namespace fo
