// The balanced router: a token's experts and weights (moe_scores.cuh), and the row
// tables, a stable counting sort of the (token, slot) pairs by expert:
//   row(t, s) = first[e] + |{(t', s') before (t, s): id(t', s') = e}|.
//
// One kernel.  CTA c owns a contiguous chunk of tokens, a warp one or two at a time:
//   1. choose; ids stay in shared memory; the CTA's share of the tables is emptied;
//   2. count the chunk's pairs per expert and segment (32 pairs or a multiple);
//   3. grid barrier, with every chunk's counts in global memory;
//   4. the experts' ranges and this chunk's start in each, then the pairs' rows.
// Up to 16 tokens, one per warp of a CTA, need no barrier: then every CTA
// makes the same choice, and each fills its share of the tables (of one token over
// 128 experts these are 130 KB, more than one CTA should write).
//
// Bytes are few (a logit once); instructions bound it.  16384 tokens of 256 experts in 8
// groups, top 8, take 32 us on the device: 18 of choosing, with about 900 warp
// instructions a token and about two thirds of the issue slots in use, up to 5 more in a
// CTA with a token to decide in fp64, 1.5 to begin, and 6 of barrier, counts and rows.
// One token takes 8.
#include <cuda_runtime.h>

#include <mutex>

#include "moe_scores.cuh"

namespace fo {

namespace {

constexpr int kScoredSmemLimit = 200 * 1024;   // that a launch asks for
constexpr int kScoredMaxCtas = 256;            // whose counts the workspace has room for
constexpr int kShareRows = 4096;               // of the tables, per CTA without a barrier

struct ScoredArgs {
  ScoreArgs score;
  int32_t tokens;
  int64_t capacity, table_rows;
  int32_t* ids;
  float* weights;
  int32_t* row_token;
  int32_t* row_slot;
  int32_t* token_row;
  int32_t* expert_first;
  int32_t* expert_rows;
  uint32_t* barrier;   // [0] count, [1] leave
  void* counts;        // [grid][pitch] pairs of each chunk per expert, 16 bits each
                       //   where a chunk has fewer tokens than that holds, else 32
  int32_t* status;
  int32_t chunk;       // tokens per CTA
  int32_t segments;    // of a chunk's pairs
  int32_t pitch;       // experts, to a multiple of 8
  int32_t alone;       // every CTA has all tokens, and there is no barrier
};

constexpr int kScoredThreads = 512;            // 128 registers each

__device__ __forceinline__ void clear_rows(int32_t* p, int64_t lo, int64_t hi, int32_t v) {
  if (((reinterpret_cast<uintptr_t>(p + lo)) & 15) == 0) {
    const int64_t n = (hi - lo) / 4;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x)
      reinterpret_cast<int4*>(p + lo)[i] = make_int4(v, v, v, v);
    lo += n * 4;
  }
  for (int64_t i = lo + threadIdx.x; i < hi; i += blockDim.x) p[i] = v;
}

// KEPT: the chunk's ids stay in shared memory, where they fit.
template <int V, bool KEPT>
__global__ void __launch_bounds__(kScoredThreads, 1) scored_kernel(const ScoredArgs a) {
  extern __shared__ int32_t sm[];
  const int E = a.score.experts, K = a.score.top_k;
  int32_t* cnt = KEPT ? sm + int64_t(a.chunk) * K : sm;   // [segments][E]
  int32_t* start = cnt + a.segments * E;                  // [E] of this chunk
  int32_t* total = start + E;                             // [E]
  int32_t* first = total + E;                             // [E]
  __shared__ int32_t ok_s;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = int(blockDim.x) / 32;
  const bool lead = !a.alone || blockIdx.x == 0;          // this CTA writes its tokens' outputs
  const int64_t t0 = a.alone ? 0 : int64_t(blockIdx.x) * a.chunk;
  const int n = int(min(int64_t(a.chunk), int64_t(a.tokens) - t0));
  const int pairs = n * K;
  int32_t* ids = KEPT ? sm : a.ids + t0 * K;              // [chunk * K]
  // a segment's pairs, whole groups of 32
  const int per = (pairs + a.segments * 32 - 1) / (a.segments * 32) * 32;
  // a warp takes kTokens tokens at a time, and the next ones' logits are on their way
  // meanwhile, where it has registers for that
  const LaneExperts<V> own(a.score);
  constexpr int kTokens = V <= 8 ? 2 : 1;
  constexpr bool kAhead = V <= 8;
  float ahead[kTokens][V];
  const auto load = [&](int t) {
#pragma unroll
    for (int j = 0; j < kTokens; ++j)
      own.load(a.score, (t0 + t + j * warps) * a.score.stride, t + j * warps < n, ahead[j]);
  };
  if constexpr (kAhead) load(warp);
  for (int i = threadIdx.x; i < (a.segments + 2) * E; i += blockDim.x) cnt[i] = 0;
  // this CTA's share of the row tables starts empty
  const int64_t share = ((a.table_rows + gridDim.x - 1) / gridDim.x + 3) / 4 * 4;
  const int64_t lo = min(share * blockIdx.x, a.table_rows), hi = min(lo + share, a.table_rows);
  clear_rows(a.row_token, lo, hi, -1);
  clear_rows(a.row_slot, lo, hi, 0);
  for (int t = warp; t < n; t += kTokens * warps) {
    int64_t at[kTokens];
    float x[kTokens][V], w[kTokens];
    int id[kTokens];
    if constexpr (!kAhead) load(t);
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      // (of a token past the last, the first is looked at once more where it must be)
      at[j] = (t0 + (t + j * warps < n ? t + j * warps : t)) * a.score.stride;
#pragma unroll
      for (int i = 0; i < V; ++i) x[j][i] = ahead[j][i];
    }
    if constexpr (kAhead) load(t + kTokens * warps);
    warp_choose<V, kTokens>(a.score, own, at, x, id, w);
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      const int u = t + j * warps;
      if (u >= n || lane >= K) continue;
      ids[u * K + lane] = id[j];
      if (lead) {
        a.ids[(t0 + u) * K + lane] = id[j];
        a.weights[(t0 + u) * K + lane] = w[j];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
    const int e = ids[i];
    if (e >= 0) atomicAdd(&cnt[(i / per) * E + e], 1);
  }
  __syncthreads();
  // per expert: the chunk's total, and each segment's start inside the chunk
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int sum = 0;
    for (int w = 0; w < a.segments; ++w) {
      const int c = cnt[w * E + e];
      cnt[w * E + e] = sum;
      sum += c;
    }
    if (a.alone)
      total[e] = sum;
    else if (a.chunk <= 65535)
      __stcg(static_cast<uint16_t*>(a.counts) + blockIdx.x * a.pitch + e, uint16_t(sum));
    else
      __stcg(static_cast<int32_t*>(a.counts) + blockIdx.x * E + e, sum);
  }
  if (!a.alone) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) ok_s = grid_barrier(a.barrier, gridDim.x, a.status);
    __syncthreads();
    if (threadIdx.x == 0) grid_barrier_leave(a.barrier + 1, a.barrier, 1, gridDim.x);
    if (!ok_s) return;
    // earlier chunks' pairs per expert and the total.  152 CTAs read 152 rows of counts
    // each: in 16 bits, eight experts per load, the threads of a column sharing out
    // the rows (one 32-bit count per load: 16384 x 256 took 5 us longer).
    if (a.chunk <= 65535) {
      const int columns = a.pitch / 8, parts = max(int(blockDim.x) / columns, 1);
      for (int i = threadIdx.x; i < columns * parts; i += blockDim.x) {
        const int col = i % columns;
        uint32_t before[4] = {0, 0, 0, 0}, all[4] = {0, 0, 0, 0};     // two experts each:
        int hi_before[4] = {0, 0, 0, 0}, hi_all[4] = {0, 0, 0, 0};    // low halves, high halves
        const uint4* row = static_cast<const uint4*>(a.counts) + col;
        constexpr int kRows = 10;       // at a time: 152 CTAs' 256 experts at once
        for (int c0 = i / columns; c0 < int(gridDim.x); c0 += kRows * parts) {
          uint4 v[kRows];
#pragma unroll
          for (int k = 0; k < kRows; ++k) {
            const int c = c0 + k * parts;
            v[k] = c < int(gridDim.x) ? __ldcg(row + c * columns) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int k = 0; k < kRows; ++k) {
            const bool earlier = c0 + k * parts < int(blockIdx.x);
            const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              all[j] += u[j] & 0xffffu;
              hi_all[j] += int(u[j] >> 16);
              before[j] += earlier ? u[j] & 0xffffu : 0u;
              hi_before[j] += earlier ? int(u[j] >> 16) : 0;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = col * 8 + 2 * j;
          // (integers: in any order)
          if (e < E && all[j]) atomicAdd(&total[e], int(all[j]));
          if (e < E && before[j]) atomicAdd(&start[e], int(before[j]));
          if (e + 1 < E && hi_all[j]) atomicAdd(&total[e + 1], hi_all[j]);
          if (e + 1 < E && hi_before[j]) atomicAdd(&start[e + 1], hi_before[j]);
        }
      }
    } else {
      for (int e = threadIdx.x; e < E; e += blockDim.x) {
        const int32_t* row = static_cast<const int32_t*>(a.counts) + e;
        int before = 0, all = 0;
        for (int c = 0; c < int(gridDim.x); ++c) {
          const int v = __ldcg(row + c * E);
          before += c < int(blockIdx.x) ? v : 0;
          all += v;
        }
        total[e] = all;
        start[e] = before;
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    // a lane takes consecutive experts
    const int q = (E + 31) / 32;
    int span = 0;
    for (int e = lane * q; e < min((lane + 1) * q, E); ++e) span += (total[e] + 127) & ~127;
    int at = span;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += v;
    }
    at -= span;
    for (int e = lane * q; e < min((lane + 1) * q, E); ++e) {
      const int rows = total[e];
      const int f = a.capacity ? int(int64_t(e) * a.capacity) : at;
      first[e] = f;
      at += (rows + 127) & ~127;
      if (blockIdx.x == 0) {
        a.expert_first[e] = f;
        a.expert_rows[e] = a.capacity ? int(min(int64_t(rows), a.capacity)) : rows;
      }
    }
  }
  __syncthreads();
  // place the pairs: rank inside the segment by a match of 32
  for (int w = warp; w < a.segments; w += warps) {
    int32_t* run = cnt + w * E;
    const int end = min((w + 1) * per, pairs);
    for (int i0 = w * per; i0 < end; i0 += 32) {
      const int i = i0 + lane;
      const int e = i < end ? ids[i] : -1;
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
      if (i < end) {
        if (lead) a.token_row[t0 * K + i] = row;
        if (row >= 0 && (!a.alone || (row >= lo && row < hi))) {
          a.row_token[row] = int32_t(t0 + i / K);
          a.row_slot[row] = i % K;
        }
      }
    }
  }
}

int64_t scored_smem(int64_t kept, int experts, int segments) {
  return 4 * (kept + int64_t(segments + 3) * experts);
}

template <int V, bool KEPT>
fo_status launch_as(const ScoredArgs& a, int grid, int smem, cudaStream_t st) {
  // the limit once, not each launch's size: another thread's launch may follow
  static std::once_flag once[64];
  static cudaError_t err[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FO_ERR_CUDA;
  const int slot = dev < 64 ? dev : 63;
  std::call_once(once[slot], [&] {
    err[slot] = cudaFuncSetAttribute(scored_kernel<V, KEPT>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kScoredSmemLimit);
  });
  if (err[slot] != cudaSuccess) return FO_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kScoredThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.alone ? 0 : 1;
  if (cudaLaunchKernelEx(&cfg, scored_kernel<V, KEPT>, a) != cudaSuccess) {
    cudaGetLastError();
    return FO_ERR_CUDA;
  }
  return FO_OK;
}

template <int V>
fo_status launch_v(ScoredArgs a, int sms, cudaStream_t st) {
  constexpr int warps = kScoredThreads / 32;
  const int E = a.score.experts, K = a.score.top_k;
  a.score.vec = a.score.vec && a.score.per % V == 0 && V * (a.score.bf16 ? 2 : 4) % 16 == 0;
  int64_t grid;
  a.alone = a.tokens <= warps;
  if (a.alone) {
    a.chunk = a.tokens;
    grid = (a.table_rows + kShareRows - 1) / kShareRows;
    if (grid > sms) grid = sms;
    if (grid < 1) grid = 1;
  } else {
    // at least a warp's worth each, and no more CTAs than SMs, so that the barrier's
    // grid is resident at once
    if (sms > kScoredMaxCtas) sms = kScoredMaxCtas;
    int64_t chunk = (int64_t(a.tokens) + sms - 1) / sms;
    if (chunk < warps) chunk = warps;
    a.chunk = int32_t(chunk);
    grid = (a.tokens + chunk - 1) / chunk;
  }
  const int64_t groups = (int64_t(a.chunk) * K + 31) / 32;
  a.segments = int32_t(groups < 1 ? 1 : groups < warps ? groups : warps);
  const int64_t kept = scored_smem(int64_t(a.chunk) * K, E, a.segments);
  if (kept <= kScoredSmemLimit) return launch_as<V, true>(a, int(grid), int(kept), st);
  return launch_as<V, false>(a, int(grid), int(scored_smem(0, E, a.segments)), st);
}

}  // namespace

fo_status launch_moe_route_scored(const fo_route_desc& d, const void* logits, fo_type type,
                                  int64_t tokens, int64_t row_stride, const float* bias,
                                  int64_t table_rows, int32_t* ids, float* weights,
                                  int32_t* row_token, int32_t* row_slot, int32_t* token_row,
                                  int32_t* expert_first, int32_t* expert_rows, void* workspace,
                                  int32_t* dev_status, void* stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FO_ERR_CUDA;
  ScoredArgs a{};
  ScoreArgs& s = a.score;
  s.logits = logits;
  s.stride = row_stride;
  s.bias = bias;
  s.bf16 = type == FO_TYPE_BF16;
  s.experts = d.experts;
  s.top_k = d.top_k;
  s.renormalize = d.renormalize != 0;
  s.sigmoid = d.score == FO_SCORE_SIGMOID;
  s.groups = d.groups;
  s.top_groups = d.top_groups;
  s.group_top = d.group_top;
  s.per = d.experts / d.groups;
  s.scale = d.scale;
  s.lane_bits = 5;
  while ((d.groups << s.lane_bits) > 32) --s.lane_bits;
  const int64_t size = s.bf16 ? 2 : 4;
  s.vec = ((reinterpret_cast<uintptr_t>(logits) | uintptr_t(row_stride * size)) & 15) == 0;
  a.tokens = int32_t(tokens);
  a.capacity = d.capacity;
  a.table_rows = table_rows;
  a.ids = ids;
  a.weights = weights;
  a.row_token = row_token;
  a.row_slot = row_slot;
  a.token_row = token_row;
  a.expert_first = expert_first;
  a.expert_rows = expert_rows;
  a.barrier = static_cast<uint32_t*>(workspace);
  a.counts = static_cast<uint8_t*>(workspace) + 256;
  a.pitch = (d.experts + 7) / 8 * 8;
  a.status = dev_status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // a lane's experts: of a group, and up to 64 (a group of 60 to a lane)
  const int v = (s.per + (1 << s.lane_bits) - 1) >> s.lane_bits;
  if (v <= 1) return launch_v<1>(a, sms, st);
  if (v <= 2) return launch_v<2>(a, sms, st);
  if (v <= 4) return launch_v<4>(a, sms, st);
  if (v <= 8) return launch_v<8>(a, sms, st);
  if (v <= 16) return launch_v<16>(a, sms, st);
  if (v <= 32) return launch_v<32>(a, sms, st);
  return launch_v<64>(a, sms, st);
}

}  // namespace fo
