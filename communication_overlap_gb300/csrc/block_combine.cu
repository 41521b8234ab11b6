// The weighted sum of a token's rows of the experts' outputs, and its gradients.
//
//   y_t = sum over slots s of w_ts rows[r_ts],  r = token_row (-1: no row)
//   drows[r_ts] = w_ts dy_t,  dw_ts = <dy_t, rows[r_ts]>,  drows = 0 elsewhere.
//
// Both move each byte once and HBM bounds them: 16384 x 4096 of bf16, top 2, 403 MB in
// 66 us (6.1 TB/s) and back 680 MB in 105 (6.5); 5001 x 2048 of fp32, top 6, 265 MB in
// 42 us (6.3) and 517 MB in 84 (6.1).  Sums are fp32, in slot order; outputs are rounded
// once.
#include <cuda_runtime.h>

#include "block_common.cuh"

namespace fo {

namespace {

constexpr int kThreads = 256;

struct CombineArgs {
  const void* rows;
  int64_t row_stride, table_rows;
  const int32_t* token_row;
  const float* weights;    // NULL: ones
  int32_t tokens, hidden, top_k;
  void* y;
  int64_t y_stride;
  int32_t* status;
  // the shape of the work: an item is `per_item` tokens' columns of one piece
  int32_t pieces;          // items along a token's columns
  int32_t per_item;
  int32_t chunks;          // threads along a token's columns
  int32_t items;
  int32_t side_by_side;    // two neighbouring lanes' eights lie next to each other in y
};

// The row of a pair, -1 for none; a row outside the table is recorded.
__device__ __forceinline__ int row_of(int32_t r, int64_t table_rows, int32_t* status) {
  if (r < table_rows) return r;
  atomicCAS(status, 0, int32_t(FO_ERR_ARG));
  return -1;
}

// Rows on 16 bytes: a thread takes eight columns of TOKENS tokens, SLOTS of their slots
// at a time.  CTAs walk over the items, and the next item's rows are looked up while
// this one's are on their way: a look-up and the rows it names are two waits in a row
// otherwise.  Of bf16 rows four CTAs fit on an SM (16384 x 4096, top 2, 66.5 us; three
// 69); fp32 rows' registers would spill (106 -> 151).
template <typename T, typename O, int SLOTS, int TOKENS>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 1)
    combine_kernel(const CombineArgs a) {
  const int local = a.pieces > 1 ? 0 : int(threadIdx.x) / a.chunks;
  const int lane_col = a.pieces > 1 ? int(threadIdx.x) : int(threadIdx.x) % a.chunks;
  const int per = a.per_item / TOKENS;      // from one of the thread's tokens to the next
  int32_t r[TOKENS][SLOTS];
  float w[TOKENS][SLOTS];
  const auto token = [&](int item, int i) {
    return int64_t(item / a.pieces) * a.per_item + local + i * per;
  };
  const auto column = [&](int item) {
    return (int64_t(item % a.pieces) * kThreads + lane_col) * 8;
  };
  const auto look_up = [&](int item, int s0) {
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
      const int64_t t = token(item, i);
      const bool live = item < a.items && local < per && t < a.tokens;
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) {
        const bool has = live && s0 + j < a.top_k;
        r[i][j] = has ? __ldg(a.token_row + t * a.top_k + s0 + j) : -1;
        w[i][j] = has && a.weights ? __ldg(a.weights + t * a.top_k + s0 + j) : 1.0f;
      }
    }
  };
  look_up(blockIdx.x, 0);
  for (int item = blockIdx.x; item < a.items; item += gridDim.x) {
    const int64_t col = column(item);
    const bool in = col < a.hidden;
    const T* rows = static_cast<const T*>(a.rows) + col;
    float acc[TOKENS][8];
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[i][k] = 0.0f;
    }
    for (int s0 = 0; s0 < a.top_k; s0 += SLOTS) {
      Pack8<T> v[TOKENS][SLOTS];
      float by[TOKENS][SLOTS];
      bool has[TOKENS][SLOTS];
#pragma unroll
      for (int i = 0; i < TOKENS; ++i) {
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
          const int row = r[i][j] < 0 ? -1 : row_of(r[i][j], a.table_rows, a.status);
          has[i][j] = in && row >= 0;
          by[i][j] = w[i][j];
          if (has[i][j]) v[i][j].load_once(rows + row * a.row_stride);
        }
      }
      if (s0 + SLOTS < a.top_k)
        look_up(item, s0 + SLOTS);
      else
        look_up(item + gridDim.x, 0);
#pragma unroll
      for (int i = 0; i < TOKENS; ++i) {
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
          if (has[i][j]) {
            float f[8];
            v[i][j].get(f);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[i][k] = fmaf(by[i][j], f[k], acc[i][k]);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
      const int64_t t = token(item, i);
      const bool live = in && local < per && t < a.tokens;
      O* to = static_cast<O*>(a.y) + t * a.y_stride + col;
      if (sizeof(O) == 2 || a.side_by_side)
        store8_warp(to, live, acc[i]);
      else if (live)
        store8(to, acc[i]);
    }
  }
}

// Any rows: a warp takes kUnits times 32 E columns of a token, a lane E neighbouring
// ones of each 32 E (one column of two tokens per thread: 245 us for 16384 x 4095 of
// bf16, top 1, where rows on 16 bytes take 35).
constexpr int kUnits = 4;
template <typename T, typename O, int E>
__global__ void __launch_bounds__(kThreads) combine_any_kernel(const CombineArgs a) {
  constexpr int kSlots = 4;
  const int64_t item = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = item / a.pieces;
  if (t >= a.tokens) return;
  const int lane = threadIdx.x & 31;
  const int first = int(item % a.pieces) * kUnits * 32 * E + lane * E;
  const T* rows = static_cast<const T*>(a.rows) + first;
  float acc[kUnits][E];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
#pragma unroll
    for (int e = 0; e < E; ++e) acc[i][e] = 0.0f;
  }
  for (int s0 = 0; s0 < a.top_k; s0 += kSlots) {
    int r[kSlots];
    float w[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      const bool has = s0 + j < a.top_k;
      r[j] = has ? __ldg(a.token_row + t * a.top_k + s0 + j) : -1;
      w[j] = has && a.weights ? __ldg(a.weights + t * a.top_k + s0 + j) : 1.0f;
    }
    Few<T, E> v[kSlots][kUnits];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      if (r[j] >= 0) r[j] = row_of(r[j], a.table_rows, a.status);
      if (r[j] < 0) continue;
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
        if (first + i * 32 * E < a.hidden) v[j][i].load(rows + r[j] * a.row_stride + i * 32 * E);
    }
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      if (r[j] < 0) continue;
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        float x[E];
        v[j][i].get(x);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[i][e] = fmaf(w[j], x[e], acc[i][e]);
      }
    }
  }
  O* y = static_cast<O*>(a.y) + t * a.y_stride + first;
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
    if (first + i * 32 * E < a.hidden) Few<O, E>::store(y + i * 32 * E, acc[i]);
}

struct CombineBackArgs {
  CombineArgs f;
  const void* dy;
  int64_t dy_stride;
  const int32_t* row_token;
  void* drows;
  int64_t drows_stride;
  float* dweights;
  int32_t warps;            // of a token: 1, 2, 4 or 8
};

// The rows that hold no token become zeros: a warp looks at up to 32 of them, far apart,
// as they come in runs, and at few where there are few (256 tokens of 4096 with 1024
// empty rows: 32 each 27 us, so 7; 5 of 4271, 60 experts of which most rows are empty,
// 70 and 26).  Rows need not lie on 16 bytes.
template <typename T>
__device__ __forceinline__ void zero_empty_rows(const CombineBackArgs& a) {
  constexpr int kOf16 = 16 / int(sizeof(T));
  const int lane = threadIdx.x & 31;
  const int warps = int(gridDim.x) * (kThreads / 32), rows = int(a.f.table_rows);
  const int each = min(32, (rows - 1) / warps + 1), looks = (rows - 1) / each + 1;
  for (int i = int(blockIdx.x) * (kThreads / 32) + int(threadIdx.x >> 5); i < looks; i += warps) {
    const int64_t row = i + int64_t(lane) * looks;
    uint32_t todo =
        __ballot_sync(0xffffffffu, lane < each && row < rows && __ldg(a.row_token + row) < 0);
    for (; todo; todo &= todo - 1) {
      T* at = static_cast<T*>(a.drows) + (i + int64_t(__ffs(todo) - 1) * looks) * a.drows_stride;
      // up to the first 16 bytes, in wide stores, and the rest
      const int head = min(int((16 - (reinterpret_cast<uintptr_t>(at) & 15)) & 15) / int(sizeof(T)),
                           a.f.hidden);
      const int wide = (a.f.hidden - head) / kOf16, tail = (a.f.hidden - head) % kOf16;
      if (lane < head) at[lane] = T(0);
      at += head;
      for (int c = lane; c < wide; c += 32)
        __stcs(reinterpret_cast<uint4*>(at) + c, make_uint4(0, 0, 0, 0));
      if (lane < tail) at[wide * kOf16 + lane] = T(0);
    }
  }
}

// The rounds of a group of warps: SLOTS slots of a token at a time.
template <int SLOTS>
struct Round {
  int64_t t;
  int s0;
  __device__ __forceinline__ void advance(const CombineArgs& f, int64_t step) {
    s0 += SLOTS;
    if (s0 >= f.top_k) s0 = 0, t += step;
  }
};

// A lane's slot of a round: its row and weight.
template <int SLOTS>
__device__ __forceinline__ void look_up(const CombineArgs& f, const Round<SLOTS>& q, bool mine,
                                        int slot, int32_t& r, float& w) {
  const bool has = mine && q.t < f.tokens && q.s0 + slot < f.top_k;
  const int64_t at = q.t * f.top_k + q.s0 + slot;
  r = has ? __ldg(f.token_row + at) : -1;
  w = has && f.weights ? __ldg(f.weights + at) : 1.0f;
}

// The threads of a token meet.
__device__ __forceinline__ void meet(int group, int warps) {
  if (warps == 1)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(warps * 32) : "memory");
}

// Rows on 16 bytes.  A token belongs to a group of warps; a round is SLOTS of its
// slots, in pieces of CHUNKS times eight columns per thread: dy, the rows, their
// products and the rows' gradients.  Groups walk over the tokens, each at its own
// pace.  STAGES - 1 pieces ahead of the one that is worked on are on their way into the
// ring, and the group's first warp looks the rows up and checks them three rounds
// ahead, for all: look-up, check and rows are three waits in a row otherwise (161 us
// for 16384 x 4096, top 2; with look-ups ahead alone 136; with the ring, but eight
// warps to each token, which meet at its sums, 125).
template <typename T, typename O, int SLOTS, int CHUNKS, int STAGES>
__global__ void __launch_bounds__(kThreads, 3) combine_backward_kernel(const CombineBackArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kWarps = kThreads / 32;
  __shared__ float part[2][kWarps][SLOTS];
  __shared__ int32_t row_s[4][kWarps][SLOTS];          // of the round (by 4) and the group
  __shared__ float weight_s[4][kWarps][SLOTS];
  constexpr int kT = sizeof(T) / 2, kO = sizeof(O) / 2;     // pieces of eight columns
  constexpr int kOf = kO + SLOTS * kT, kPieces = CHUNKS * kOf;
  const CombineArgs& f = a.f;
  const OwnRing ring(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / a.warps;
  const bool leads = warp % a.warps == 0 && lane < SLOTS;
  const int per = kWarps / a.warps;                    // tokens of a CTA
  const int64_t step = int64_t(gridDim.x) * per;
  const int64_t first = int64_t(blockIdx.x) * per + group;
  const int col0 = ((warp % a.warps) * 32 + lane) * 8;
  const int stride = a.warps * 32 * 8;                 // from one of a thread's columns to the next
  const auto name = [&](int32_t r) {
    return r >= 0 && r < f.table_rows ? __ldg(a.row_token + r) : -1;
  };
  const auto publish = [&](int i, int64_t t, int32_t r, int32_t by, float w) {
    if (!leads) return;
    // (a row outside the table, or one that holds another token, is not this one's)
    if (r >= 0 && by != int32_t(t)) {
      atomicCAS(f.status, 0, int32_t(FO_ERR_ARG));
      r = -1;
    }
    row_s[i & 3][group][lane] = r;
    weight_s[i & 3][group][lane] = w;
  };
  // the rounds that are worked on, fetched next, published next and looked up next
  Round<SLOTS> now{first, 0}, ahead{first, 0}, named{first, 0}, looked{first, 0};
  int32_t r3, by3, r4;
  float w3, w4;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    look_up(f, looked, leads, lane, r3, w3);
    publish(i, looked.t, r3, name(r3), w3);
    looked.advance(f, step);
    named.advance(f, step);
  }
  look_up(f, looked, leads, lane, r3, w3);
  by3 = name(r3);
  looked.advance(f, step);
  look_up(f, looked, leads, lane, r4, w4);
  looked.advance(f, step);
  meet(group, a.warps);
  int ahead_i = 0, ahead_c = 0;
  const auto fetch = [&](int stage) {
    if (ahead.t < f.tokens) {
      int32_t r[SLOTS];
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) r[j] = row_s[ahead_i & 3][group][j];
#pragma unroll
      for (int k = 0; k < CHUNKS; ++k) {
        const int c = col0 + ahead_c + k * stride, at = stage * kPieces + k * kOf;
        if (c - lane * 8 >= f.hidden) continue;
        ring.fetch(at, static_cast<const O*>(a.dy) + ahead.t * a.dy_stride, c, f.hidden);
        if (a.dweights == nullptr) continue;
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
          if (r[j] >= 0)
            ring.fetch(at + kO + j * kT, static_cast<const T*>(f.rows) + r[j] * f.row_stride, c,
                       f.hidden);
      }
    }
    OwnRing::commit();
    ahead_c += CHUNKS * stride;
    if (ahead_c >= f.hidden) {
      ahead_c = 0;
      ++ahead_i;
      ahead.advance(f, step);
    }
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);
  int turn = 0, stage = 0;
  for (int i = 0; now.t < f.tokens; ++i) {
    int32_t r[SLOTS];
    float w[SLOTS];
    Pair dot[SLOTS];
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      r[j] = row_s[i & 3][group][j];
      w[j] = weight_s[i & 3][group][j];
      dot[j] = Pair::of(0.0f);
    }
    for (int c0 = 0; c0 < f.hidden; c0 += CHUNKS * stride) {
      fetch(stage == 0 ? STAGES - 1 : stage - 1);
      OwnRing::wait<STAGES - 1>();
#pragma unroll
      for (int k = 0; k < CHUNKS; ++k) {
        const int c = col0 + c0 + k * stride, at = stage * kPieces + k * kOf;
        if (c - lane * 8 >= f.hidden) continue;
        const bool in = c < f.hidden;
        Pair x[4], y[4];
        get_pairs<O>(ring, at, x);
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
          if (r[j] >= 0) {
            if (a.dweights && in) {
              get_pairs<T>(ring, at + kO + j * kT, y);
#pragma unroll
              for (int e = 0; e < 4; ++e) dot[j] = fma2(x[e], y[e], dot[j]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = Pair::of(w[j]) * x[e];
            store8_warp(static_cast<T*>(a.drows) + (r[j] * a.drows_stride + c), in, y);
          }
      }
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    publish(i + 3, named.t, r3, by3, w3);
    named.advance(f, step);
    r3 = r4, w3 = w4;
    by3 = name(r3);
    look_up(f, looked, leads, lane, r4, w4);
    looked.advance(f, step);
    if (a.dweights) {
      float sum[SLOTS];
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) {
        sum[j] = warp_sum(dot[j].sum());
        if (lane == 0) part[turn][warp][j] = sum[j];
      }
    }
    meet(group, a.warps);
    if (a.dweights && leads && now.s0 + lane < f.top_k) {
      float sum = 0.0f;
      for (int k = 0; k < a.warps; ++k) sum += part[turn][warp + k][lane];
      a.dweights[now.t * f.top_k + now.s0 + lane] = sum;
    }
    turn ^= 1;
    now.advance(f, step);
  }
  OwnRing::wait<0>();
  zero_empty_rows<T>(a);
}

// Any rows: E neighbouring columns per thread and 32 E, without the ring.
template <typename T, typename O, int SLOTS, int E>
__global__ void __launch_bounds__(kThreads) combine_backward_any_kernel(const CombineBackArgs a) {
  __shared__ float part[2][kThreads / 32][SLOTS];
  const CombineArgs& f = a.f;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / a.warps, per = (kThreads / 32) / a.warps;
  const int64_t step = int64_t(gridDim.x) * per;
  int turn = 0;
  Round<SLOTS> now{int64_t(blockIdx.x) * per + group, 0};
  for (; now.t < f.tokens; now.advance(f, step)) {
    int32_t mine, by;
    float weight;
    look_up(f, now, lane < SLOTS, lane, mine, weight);
    by = mine >= 0 && mine < f.table_rows ? __ldg(a.row_token + mine) : -1;
    if (mine >= 0 && by != int32_t(now.t)) {
      atomicCAS(f.status, 0, int32_t(FO_ERR_ARG));
      mine = -1;
    }
    int32_t r[SLOTS];
    float w[SLOTS], dot[SLOTS];
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      r[j] = __shfl_sync(0xffffffffu, mine, j);
      w[j] = __shfl_sync(0xffffffffu, weight, j);
      dot[j] = 0.0f;
    }
    const O* dy = static_cast<const O*>(a.dy) + now.t * a.dy_stride;
    // kUnits loads of a row before their stores
    const int stride = a.warps * 32 * E;
    for (int c0 = ((warp % a.warps) * 32 + lane) * E; c0 < f.hidden; c0 += kUnits * stride) {
      Few<O, E> g[kUnits];
      Few<T, E> v[kUnits][SLOTS];
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const int c = c0 + k * stride;
        if (c >= f.hidden) continue;
        g[k].load(dy + c);
        if (a.dweights == nullptr) continue;
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
          if (r[j] >= 0) v[k][j].load(static_cast<const T*>(f.rows) + (r[j] * f.row_stride + c));
      }
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const int c = c0 + k * stride;
        if (c >= f.hidden) continue;
        float x[E];
        g[k].get(x);
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
          if (r[j] >= 0) {
            float y[E];
            if (a.dweights) {
              v[k][j].get(y);
#pragma unroll
              for (int e = 0; e < E; ++e) dot[j] = fmaf(x[e], y[e], dot[j]);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = w[j] * x[e];
            Few<T, E>::store(static_cast<T*>(a.drows) + (r[j] * a.drows_stride + c), y);
          }
      }
    }
    if (a.dweights == nullptr) continue;
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      dot[j] = warp_sum(dot[j]);
      if (lane == 0) part[turn][warp][j] = dot[j];
    }
    meet(group, a.warps);
    if (warp % a.warps == 0 && lane < SLOTS && now.s0 + lane < f.top_k) {
      float sum = 0.0f;
      for (int k = 0; k < a.warps; ++k) sum += part[turn][warp + k][lane];
      a.dweights[now.t * f.top_k + now.s0 + lane] = sum;
    }
    turn ^= 1;
  }
  zero_empty_rows<T>(a);
}

// How many CTAs of a kernel, with so much shared memory always, the device holds at
// once; asked for once per device.
template <auto K>
fo_status resident(int smem, int* ctas) {
  static std::once_flag once[64];
  static int count[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FO_ERR_CUDA;
  const fo_status q = smem > 0 ? allow_smem<K>() : FO_OK;
  if (q != FO_OK) return q;
  const int slot = dev < 64 ? dev : 63;
  std::call_once(once[slot], [&] {
    int per_sm = 0, sms = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, K, kThreads, smem) == cudaSuccess &&
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
      count[slot] = per_sm * sms;
  });
  *ctas = count[slot];
  return count[slot] > 0 ? FO_OK : FO_ERR_CUDA;
}

template <typename T, typename O, int SLOTS, int TOKENS>
fo_status forward_as(CombineArgs a, cudaStream_t st) {
  const int64_t chunks = a.hidden / 8;
  a.pieces = int32_t((chunks + kThreads - 1) / kThreads);
  a.chunks = int32_t(chunks < kThreads ? chunks : kThreads);
  a.per_item = (a.pieces > 1 ? 1 : kThreads / a.chunks) * TOKENS;
  const int64_t items = (int64_t(a.tokens) + a.per_item - 1) / a.per_item * a.pieces;
  if (items >= (int64_t(1) << 30)) return FO_ERR_UNSUPPORTED;
  a.items = int32_t(items);
  // (of an odd number of eights every other token's last has the next one's first beside it,
  // which follows in memory only where the rows are not padded)
  a.side_by_side = a.pieces > 1 || a.chunks % 2 == 0 || a.y_stride == a.hidden;
  constexpr auto kernel = combine_kernel<T, O, SLOTS, TOKENS>;
  int ctas = 0;
  const fo_status q = resident<kernel>(0, &ctas);
  if (q != FO_OK) return q;
  kernel<<<unsigned(items < ctas ? items : ctas), kThreads, 0, st>>>(a);
  return FO_OK;
}

template <typename T, typename O, int E>
fo_status forward_any(CombineArgs a, cudaStream_t st) {
  a.pieces = (a.hidden + kUnits * 32 * E - 1) / (kUnits * 32 * E);
  const int64_t grid = (int64_t(a.tokens) * a.pieces + kThreads / 32 - 1) / (kThreads / 32);
  if (grid >= (int64_t(1) << 31)) return FO_ERR_UNSUPPORTED;
  combine_any_kernel<T, O, E><<<unsigned(grid), kThreads, 0, st>>>(a);
  return FO_OK;
}

// How all of a call's rows lie: on 16 bytes and eight columns, on two elements, or not.
enum class Rows { kEight, kTwo, kOne };

template <typename T, typename O>
fo_status forward(const CombineArgs& a, Rows rows, cudaStream_t st) {
  if (rows == Rows::kOne) return forward_any<T, O, 1>(a, st);
  if (rows == Rows::kTwo) return forward_any<T, O, 2>(a, st);
  // (16384 x 4096, top 1: as half of two slots 56 us, of fp32 77; so 49 and 65)
  if (a.top_k == 1) return forward_as<T, O, 1, 2>(a, st);
  if (a.top_k == 2) return forward_as<T, O, 2, 2>(a, st);
  return forward_as<T, O, 4, 1>(a, st);
}

// The warps of a token: the fewest (they meet at each of its sums) with which the
// groups of all CTAs come out even over the tokens to within a twentieth, or the most
// even number, up to a warp per `width` columns.
int token_warps(int64_t tokens, int64_t hidden, int width, int ctas) {
  int best = 1;
  double most = 0.0;
  for (int w = 1; w <= 8; w *= 2) {
    if (w > 1 && int64_t(w / 2) * width >= hidden) break;
    const int64_t groups = int64_t(ctas) * (kThreads / 32) / w;
    const int64_t rounds = (tokens + groups - 1) / groups;
    const double even = rounds > 0 ? double(tokens) / double(groups * rounds) : 1.0;
    if (even > most) best = w, most = even;
    if (even > 0.95) break;
  }
  return best;
}

template <auto K>
fo_status backward_as(CombineBackArgs a, int smem, int width, cudaStream_t st) {
  int ctas = 0;
  const fo_status q = resident<K>(smem, &ctas);
  if (q != FO_OK) return q;
  a.warps = token_warps(a.f.tokens, a.f.hidden, width, ctas);
  const int64_t per = (kThreads / 32) / a.warps;
  int64_t grid = (int64_t(a.f.tokens) + per - 1) / per;
  // (two rows to look at for a warp, if that many CTAs are resident)
  const int64_t looks = (a.f.table_rows + kThreads / 16 - 1) / (kThreads / 16);
  if (grid < looks) grid = looks;
  K<<<unsigned(grid < ctas ? grid : ctas), kThreads, smem, st>>>(a);
  return FO_OK;
}

// The slots of a round come out even over a token's rounds (6 as 3 and 3: 5001 x 2048
// in fp32 113 -> 89 us against 4 and 2), with two pieces of columns where few rows are
// under way in one, and as many stages as let three CTAs' rings fit on an SM.  (With fp32
// dy two fit where the rows are fp32 and a round has one slot or four, or bf16 and two.)
template <typename T, typename O, int SLOTS>
fo_status backward_slots(const CombineBackArgs& a, cudaStream_t st) {
  constexpr int kT = sizeof(T) / 2, kO = sizeof(O) / 2;
  constexpr int kChunks = SLOTS * kT <= 2 ? 2 : 1;
  constexpr int kStages = SLOTS * kT <= 4 ? 3 : 2;
  constexpr int kBytes = kStages * kChunks * (kO + SLOTS * kT) * 16 * kThreads;
  return backward_as<combine_backward_kernel<T, O, SLOTS, kChunks, kStages>>(a, kBytes, 256, st);
}

template <typename T, typename O>
fo_status backward(const CombineBackArgs& a, Rows lie, cudaStream_t st) {
  if (lie == Rows::kOne)
    return backward_as<combine_backward_any_kernel<T, O, 4, 1>>(a, 0, 32, st);
  if (lie == Rows::kTwo)
    return backward_as<combine_backward_any_kernel<T, O, 4, 2>>(a, 0, 64, st);
  const int rounds = (a.f.top_k + 3) / 4;
  switch ((a.f.top_k + rounds - 1) / rounds) {
    case 1: return backward_slots<T, O, 1>(a, st);
    case 2: return backward_slots<T, O, 2>(a, st);
    case 3: return backward_slots<T, O, 3>(a, st);
    default: return backward_slots<T, O, 4>(a, st);
  }
}

fo_status launched() { return cudaGetLastError() == cudaSuccess ? FO_OK : FO_ERR_CUDA; }

}  // namespace

fo_status launch_combine(const void* rows, fo_type type, int64_t table_rows, int64_t hidden,
                         int64_t row_stride, const int32_t* token_row, const float* weights,
                         int64_t tokens, int32_t top_k, void* y, fo_type y_type,
                         int64_t y_stride, int32_t* dev_status, void* stream) {
  CombineArgs a{};
  a.rows = rows, a.row_stride = row_stride, a.table_rows = table_rows;
  a.token_row = token_row, a.weights = weights;
  a.tokens = int32_t(tokens), a.hidden = int32_t(hidden), a.top_k = top_k;
  a.y = y, a.y_stride = y_stride, a.status = dev_status;
  const bool vec = hidden % 8 == 0 && rows_on(rows, row_stride, type, 16) &&
                   rows_on(y, y_stride, y_type, 16);
  const bool two = hidden % 2 == 0 && rows_on_two(rows, row_stride, type) &&
                   rows_on_two(y, y_stride, y_type);
  const Rows lie = vec ? Rows::kEight : two ? Rows::kTwo : Rows::kOne;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = type == FO_TYPE_BF16, ybf = y_type == FO_TYPE_BF16;
  const fo_status q = bf && ybf ? forward<uint16_t, uint16_t>(a, lie, st)
                      : bf      ? forward<uint16_t, float>(a, lie, st)
                      : ybf     ? forward<float, uint16_t>(a, lie, st)
                                : forward<float, float>(a, lie, st);
  return q == FO_OK ? launched() : q;
}

fo_status launch_combine_backward(const void* dy, fo_type dy_type, int64_t dy_stride,
                                  const void* rows, fo_type type, int64_t table_rows,
                                  int64_t hidden, int64_t row_stride, const int32_t* token_row,
                                  const int32_t* row_token, const float* weights,
                                  int64_t tokens, int32_t top_k, void* drows,
                                  int64_t drows_stride, float* dweights, int32_t* dev_status,
                                  void* stream) {
  CombineBackArgs a{};
  CombineArgs& f = a.f;
  f.rows = rows, f.row_stride = row_stride, f.table_rows = table_rows;
  f.token_row = token_row, f.weights = weights;
  f.tokens = int32_t(tokens), f.hidden = int32_t(hidden), f.top_k = top_k;
  f.status = dev_status;
  a.dy = dy, a.dy_stride = dy_stride, a.row_token = row_token;
  a.drows = drows, a.drows_stride = drows_stride, a.dweights = dweights;
  const bool vec = hidden % 8 == 0 && (!dweights || rows_on(rows, row_stride, type, 16)) &&
                   rows_on(dy, dy_stride, dy_type, 16) && rows_on(drows, drows_stride, type, 16);
  const bool two = hidden % 2 == 0 && (!dweights || rows_on_two(rows, row_stride, type)) &&
                   rows_on_two(dy, dy_stride, dy_type) && rows_on_two(drows, drows_stride, type);
  const Rows lie = vec ? Rows::kEight : two ? Rows::kTwo : Rows::kOne;
  if (tokens == 0 && table_rows == 0) return FO_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = type == FO_TYPE_BF16, ybf = dy_type == FO_TYPE_BF16;
  const fo_status q = bf && ybf ? backward<uint16_t, uint16_t>(a, lie, st)
                      : bf      ? backward<uint16_t, float>(a, lie, st)
                      : ybf     ? backward<float, uint16_t>(a, lie, st)
                                : backward<float, float>(a, lie, st);
  return q == FO_OK ? launched() : q;
}

}  // namespace fo
