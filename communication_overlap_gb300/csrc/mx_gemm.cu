// The product of two matrices in the microscaled 4-bit form, for all rows of
// A or for one range of rows per expert:
//   D[m][n] = sum_k a[m][k] b[n][k],  a[m][k] = value of the code x 2^(s - 127).
//
// The tensor cores take this form as it is (tcgen05.mma kind::mxf4 with block
// scales): codes from shared memory, scales from tensor memory, sums in fp32
// in tensor memory.  Nothing is decoded, so a value costs 4.25 bits on its
// whole way from HBM.
//
// One persistent kernel, one CTA (or CTA pair) per SM (or pair of SMs):
//  * warps 0 and 10: TMA producers.  A stage is 256 columns: 128 rows of A and
//    this CTA's rows of B, 128 bytes each (one 128-byte swizzle atom), from warp
//    0, and the scales of both, in the blocks of 512 bytes that the form keeps
//    them in, from warp 10.  (One thread for all four copies needs 600 cycles
//    per stage, as long as the MMAs.)
//  * warp 1: four MMAs of 64 columns per stage, from one thread.
//  * warps 2-5: epilogue.  Sums to bf16 or fp32, transposed through shared
//    memory so that a row's stores are whole 128-byte segments.
//  * warps 6-9: the stages' scales from shared to tensor memory, through
//    registers (tcgen05.st, a quarter of the lanes per warp), a slot per stage.
//    tcgen05.cp does the same from the MMA's thread, but in line with the MMAs:
//    the 8-expert product of 32768 x 14336 x 4096 took 1163 us with it.
// The PAIR form computes 256 x BN with one cta_group::2 MMA: each CTA holds
// 128 rows of A, half of B's rows and all of B's scales.
//
// Tensor memory: two sums of BN columns and five slots of scales in 512
// columns.  BN = 256 leaves room for 392 columns of sums, so the second sum
// starts at column 136 and shares 120 columns with the first: the epilogue
// drains a tile's 128 columns on that side first, and the next tile's MMAs wait
// for those only.
//
// What bounds it: a stage of the PAIR form brings 35 KB into an SM, 550 cycles at
// the 64 bytes per cycle that L2 delivers to one, and its MMAs take 512; of a
// tile's 10100 cycles at K = 4096 about 1150 are the wait for the shared columns.
// Narrower tiles need no sharing but more bytes per product: the 8-expert product
// below takes 609 us with 192 columns and 806 with 128, and a sixth stage changes
// neither.  Nor do scales in a ring of their own, ahead of the codes, or a second
// set of epilogue warps.
//
// Measured: 552 us in a short run and up to 630 in a long one for 32768 rows over 8
// experts, N = 14336, K = 4096 (7.0 to 6.1 PFLOP/s, at the 1.67 GHz and below that
// the power limit leaves), 44 us for 8192 x 4096 x 2752 with fp32 output (writing
// that alone takes 21), 10.4 us for 512 x 4096 x 4096.
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "moe_internal.h"
#include "mx_common.cuh"
#include "tensor_core.cuh"
#include "tensor_map.h"

namespace fo {

namespace {

constexpr int kThreads = 352;
constexpr int kStageCols = 256;                  // columns of K per stage
constexpr int kABytes = 128 * 128;
constexpr int kBBytes = 128 * 128;               // room for this CTA's rows of B
constexpr int kSaBytes = 1024;                   // 128 rows x 8 scales
constexpr int kSbBlocks = 2;                     // blocks of rows of B's scales
constexpr int kSbBytes = kSbBlocks * 1024;
constexpr int kStageBytes = kABytes + kBBytes + kSaBytes + kSbBytes;
constexpr int kStages = 5;
constexpr int kSfCols = 8 + 8 * kSbBlocks;       // columns of a slot: A's, then B's
constexpr int kSf0 = 512 - kStages * kSfCols;     // one slot per stage
constexpr int kStagingBytes = 4 * 2 * 32 * 128;    // two buffers per epilogue warp
constexpr int kStartOffset = kStages * kStageBytes + kStagingBytes;
constexpr int kBarOffset = kStartOffset + 4 * (kRouteExperts + 4);
constexpr int kSmemBytes = 1024 + kBarOffset + 256;
constexpr int kBand = 16;                        // tile rows walked per column
static_assert(kSmemBytes <= 232448, "shared memory budget");

struct GemmArgs {
  CUtensorMap map_a, map_b, map_sa, map_sb, map_d;
  const int32_t* first;
  const int32_t* rows;
  void* d;
  int64_t stride;
  int32_t M, N, n_pad, n_groups, grouped;
  int32_t k_stages, k_steps;   // stages of 256 columns, MMAs of 64 in all
  int32_t bn;                  // tile columns, a multiple of 64
  int32_t acc1;                // tensor memory column of the second sum
  int32_t vec;                 // map_d can address D's rows
  int32_t n_copied;            // a 128-byte wide copy to D may reach up to this column
  int32_t* status;
};

// kind::mxf4: A and B E2M1 (1 at bits 7 and 10), scales E8M0 (bit 23), N >> 3
// at 17, M >> 4 at 24.  The scale ids (bits 29 and 4) pick bytes 0-1 or 2-3 of
// each 32-bit cell of scales.
__device__ __forceinline__ uint32_t instruction(int m, int n) {
  return (1u << 7) | (1u << 10) | (1u << 23) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

// Wait until at most N of this thread's bulk stores still read shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// The first `rows` rows and n columns of a staging buffer to D, by a warp: by
// words, a lane each, where D's rows start on words, else by elements; eight rows
// at a time.  (Row by row, 16602 x 645 x 275 with fp32 output took 48 us and 4234
// x 3092 x 202 with bf16 41, this way 26 and 19.  Out of line: inlined, it makes
// the copies' path slower, 4234 x 3096 x 202 14.4 us instead of 12.5.)
template <bool BF16>
static __device__ __noinline__ void store_rows(uint32_t buf, uint8_t* to, int64_t pitch, int rows,
                                               int n) {
  const int lane = threadIdx.x & 31;
  const auto staged = [&](int row, int byte) {
    return buf + row * 128 + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15);
  };
  const bool words = ((reinterpret_cast<uintptr_t>(to) | uintptr_t(pitch)) & 3) == 0;
#pragma unroll 1
  for (int r = 0; r < rows; r += 8) {
    if (!BF16 || words) {
      constexpr int kPer = BF16 ? 2 : 1;       // columns of a word
      uint32_t x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x[i]) : "r"(staged(r + i, lane * 4)) : "memory");
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r + i < rows && lane * kPer + kPer <= n)
          *reinterpret_cast<uint32_t*>(to + int64_t(r + i) * pitch + lane * 4) = x[i];
      if (BF16 && (n & 1) && lane < 8 && r + lane < rows) {   // the last column
        uint16_t e;
        asm volatile("ld.shared.u16 %0, [%1];"
                     : "=h"(e) : "r"(staged(r + lane, (n - 1) * 2)) : "memory");
        *reinterpret_cast<uint16_t*>(to + int64_t(r + lane) * pitch + (n - 1) * 2) = e;
      }
    } else {
#pragma unroll
      for (int h = 0; h < 64; h += 32) {
        uint16_t x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          asm volatile("ld.shared.u16 %0, [%1];"
                       : "=h"(x[i]) : "r"(staged(r + i, (h + lane) * 2)) : "memory");
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (r + i < rows && h + lane < n)
            *reinterpret_cast<uint16_t*>(to + int64_t(r + i) * pitch + (h + lane) * 2) = x[i];
      }
    }
  }
}

struct Tile {
  int32_t row0, rows;   // first row of D, rows of the tile's range from there on
  int32_t b_row, col0;  // first row of B's stack, first column of D
};

// Tile t of the launch.  Groups in order; inside a group bands of kBand tile
// rows, column by column, so that tiles that run together share rows of A and
// of B in L2.
template <bool PAIR>
__device__ __forceinline__ Tile tile_at(const GemmArgs& a, const int32_t* start, int t, int& g) {
  while (t >= start[g + 1]) ++g;
  const int first = a.grouped ? __ldg(a.first + g) : 0, rows = a.grouped ? __ldg(a.rows + g) : a.M;
  constexpr int kM = PAIR ? 256 : 128;
  const int mt = (rows + kM - 1) / kM, nt = (a.N + a.bn - 1) / a.bn;
  int i = t - start[g];
  const int band = i / (kBand * nt);
  i -= band * kBand * nt;
  const int h = min(kBand, mt - band * kBand);
  const int n = i / h, m = band * kBand + i % h;
  return Tile{first + m * kM, rows - m * kM, g * a.n_pad + n * a.bn, n * a.bn};
}

template <bool PAIR, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) mx_gemm_kernel(const __grid_constant__ GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  // 1024-byte alignment for the swizzle atoms, at the same offset in a pair
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int32_t* start = reinterpret_cast<int32_t*>(smem + kStartOffset);   // [groups + 1] tiles before
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarOffset);    // PAIR: the leader's
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + 2;                                 // PAIR: the leader's
  uint64_t* sf_full = acc_empty + 2;       // a stage's scales are in this CTA's shared memory
  uint64_t* drain = sf_full + kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x) / 32, 0), lane = threadIdx.x % 32;
  const uint32_t rank = PAIR ? tc::cluster_rank() : 0;
  constexpr int kM = PAIR ? 256 : 128;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      // a producer and four scale warps per CTA
      mbar_init(smem_u32(&full[s]), PAIR ? 10 : 5);
      mbar_init(smem_u32(&empty[s]), 1);
      mbar_init(smem_u32(&sf_full[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_empty[b]), PAIR ? 8 : 4);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (a.k_stages > 0) {
      tc::prefetch_map(&a.map_a);
      tc::prefetch_map(&a.map_b);
      tc::prefetch_map(&a.map_sa);
      tc::prefetch_map(&a.map_sb);
    }
  }
  if (warp == 1) tc::alloc<PAIR>(smem_u32(tmem_slot), 512);
  // tiles before each group; a group out of order has none and is reported
  if (warp == 2) {
    const int nt = (a.N + a.bn - 1) / a.bn;
    int before = 0;
    for (int g0 = 0; g0 < a.n_groups; g0 += 32) {
      const int g = g0 + lane;
      int tiles = 0;
      if (g < a.n_groups) {
        const int f = a.grouped ? __ldg(a.first + g) : 0;
        const int r = a.grouped ? __ldg(a.rows + g) : a.M;
        if (f < 0 || r < 0 || (f & 127) || int64_t(f) + r > a.M) {
          if (blockIdx.x == 0) atomicCAS(a.status, 0, int32_t(FO_ERR_ARG));
        } else {
          tiles = (r + kM - 1) / kM * nt;
        }
      }
      int sum = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (g < a.n_groups) start[g] = before + sum - tiles;
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) start[a.n_groups] = before;
  }
  tc::fence_before();
  __syncthreads();
  if constexpr (PAIR) tc::cluster_sync();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  const int tiles = start[a.n_groups];
  const int worker = blockIdx.x / (PAIR ? 2 : 1), workers = gridDim.x / (PAIR ? 2 : 1);
  const int b_rows = a.bn / (PAIR ? 2 : 1);    // rows of B this CTA stages
  const bool shared_cols = a.acc1 < a.bn;      // the two sums overlap

  if (warp == 0 || warp == 10) {
    // ------------------------------------------------------------ producers
    // warp 0 the codes, warp 10 the scales; as everywhere here the whole warp
    // walks the loop and one elected thread issues
    const bool codes = warp == 0;
    const bool leader = tc::elect_one();
    const uint64_t keep = tc::policy_evict_last();
    const uint32_t bytes = codes ? uint32_t(kABytes + b_rows * 128) : uint32_t(kSaBytes + kSbBytes);
    int stage = 0, g = 0;
    uint32_t phase = 0, filled = 0;    // filled: bit s, stage s was filled at least once
    bool ok = a.k_stages > 0;
    for (int t = worker; ok && t < tiles; t += workers) {
      const Tile w = tile_at<PAIR>(a, start, t, g);
      const int a_row = w.row0 + int(rank) * 128, b_row = w.b_row + int(rank) * b_rows;
      for (int kb = 0; kb < a.k_stages; ++kb) {
        ok = tc::wait_warp(smem_u32(&empty[stage]), phase ^ 1, abort_flag, a.status);
        if (!ok) break;
        const uint32_t sa = smem_u32(smem) + uint32_t(stage * kStageBytes);
        if (leader) {
          if (!codes) {
            const uint32_t bar = smem_u32(&sf_full[stage]);
            mbar_expect_tx(bar, bytes);
            tc::load_2d(sa + kABytes + kBBytes, &a.map_sa, bar, kb * 256, a_row / 128, keep);
            tc::load_2d(sa + kABytes + kBBytes + kSaBytes, &a.map_sb, bar, kb * 256, w.b_row / 128,
                        keep);
          } else if constexpr (PAIR) {
            const uint32_t bar = tc::map_to_rank(smem_u32(&full[stage]), 0);
            if (rank == 0)
              mbar_expect_tx(smem_u32(&full[stage]), bytes);
            else
              tc::expect_tx_cluster(bar, bytes);
            tc::load_2d_pair(sa, &a.map_a, bar, kb * 128, a_row, keep);
            tc::load_2d_pair(sa + kABytes, &a.map_b, bar, kb * 128, b_row, keep);
          } else {
            const uint32_t bar = smem_u32(&full[stage]);
            mbar_expect_tx(bar, bytes);
            tc::load_2d(sa, &a.map_a, bar, kb * 128, a_row, keep);
            tc::load_2d(sa + kABytes, &a.map_b, bar, kb * 128, b_row, keep);
          }
        }
        __syncwarp();
        filled |= 1u << stage;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok && a.k_stages > 0 && leader && (!codes || rank == 0)) {
      // winding down: copies already issued land before the CTA exits
      for (int s = 0; s < kStages; ++s) {
        // the parity of stage s's last fill: this pass's, or that of the one before
        const uint32_t parity = s < stage ? phase : phase ^ 1;
        if ((filled >> s) & 1u) tc::wait_drain(smem_u32(codes ? &full[s] : &sf_full[s]), parity);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the loop, so that descriptors stay in uniform
    // registers, and one elected thread issues.
    if (rank == 0 && a.k_stages > 0) {
      const uint32_t idesc = instruction(kM, a.bn);
      const uint64_t desc0 = tc::smem_desc(smem_u32(smem), 16, 1024, 2);
      const bool leader = tc::elect_one();
      int stage = 0, g = 0, i = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = worker; ok && t < tiles; t += workers, ++i) {
        const Tile w = tile_at<PAIR>(a, start, t, g);
        const int acc = i & 1;
        // the sum's columns are free: all of tile i - 2's, or, where the two
        // sums share columns, those of tile i - 1's that are shared
        const int wait_tile = shared_cols ? i - 1 : i - 2;
        if (wait_tile >= 0 && !tc::wait_warp(smem_u32(&acc_empty[acc]),
                                             uint32_t(wait_tile >> 1) & 1, abort_flag, a.status))
          break;
        const uint32_t d = tmem + uint32_t(acc ? a.acc1 : 0);
        const uint32_t b_shift = uint32_t(w.b_row % 128) / 32;   // columns of scales before b_row
        const uint32_t sf_b = 8 + b_shift, sf_half = uint32_t(kSbBlocks) * 4;
        int steps = a.k_steps;
        for (int kb = 0; kb < a.k_stages; ++kb, steps -= 4) {
          if (!tc::wait_warp(smem_u32(&full[stage]), phase, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc::fence_after();
          const uint64_t da = desc0 + uint64_t(stage * (kStageBytes >> 4));
          const uint64_t db = da + (kABytes >> 4);
          const uint32_t sfa = tmem + uint32_t(kSf0 + stage * kSfCols), sfb = sfa + sf_b;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk < steps) {
                constexpr uint32_t kHigh = (2u << 29) | (2u << 4);
                tc::mma_mxf4<PAIR>(d, da + kk * 2, db + kk * 2, (kk & 1) ? idesc | kHigh : idesc,
                                   sfa + (kk >> 1) * 4, sfb + (kk >> 1) * sf_half,
                                   (kb | kk) ? 1u : 0u);
              }
            }
            tc::commit<PAIR>(smem_u32(&empty[stage]));
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (leader) tc::commit<PAIR>(smem_u32(&acc_full[acc]));
        __syncwarp();
      }
    }
  } else if (warp >= 6 && warp < 10) {
    // ------------------------------------------------------------ scales
    const uint32_t quarter = uint32_t((warp & 3) * 32) << 16;
    const uint32_t base = smem_u32(smem) + kABytes + kBBytes + lane * 16;
    uint32_t stage = 0, phase = 0;
    bool ok = a.k_stages > 0;
    for (int t = worker; ok && t < tiles; t += workers) {
      for (int kb = 0; kb < a.k_stages; ++kb) {
        // (the stage was refilled after its last MMAs, which were also the last
        // to read its slot in tensor memory)
        ok = tc::wait_warp(smem_u32(&sf_full[stage]), phase, abort_flag, a.status);
        if (!ok) break;
        // a block of scales is 32 lanes x 16 bytes: a lane's four columns
        const uint32_t from = base + stage * kStageBytes;
        uint32_t x[2][1 + kSbBlocks][4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          tc::lds128(from + c * 512, x[c][0]);
#pragma unroll
          for (int r = 0; r < kSbBlocks; ++r)
            tc::lds128(from + kSaBytes + r * 1024 + c * 512, x[c][1 + r]);
        }
        tc::fence_after();
        const uint32_t to = tmem + quarter + uint32_t(kSf0) + stage * uint32_t(kSfCols);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          tc::tmem_st4(to + c * 4, x[c][0]);
#pragma unroll
          for (int r = 0; r < kSbBlocks; ++r)
            tc::tmem_st4(to + 8 + uint32_t(c * kSbBlocks + r) * 4, x[c][1 + r]);
        }
        tc::tmem_wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) {
          const uint32_t bar = smem_u32(&full[stage]);
          if (PAIR && rank != 0)
            tc::arrive_cluster_relaxed(tc::map_to_rank(bar, 0));
          else
            mbar_arrive(bar);
        }
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;   // this warp's quarter of the tensor memory lanes
    const uint32_t staging = smem_u32(smem + kStages * kStageBytes + (warp - 2) * (2 * 32 * 128));
    const int halves = (a.bn + 127) / 128;       // 128 columns at a time
    constexpr int es = BF16 ? 2 : 4;
    const bool zero = a.k_stages == 0;
    int g = 0, i = 0;
    uint32_t turn = 0;   // staging buffers used so far
    for (int t = worker; t < tiles; t += workers, ++i) {
      const Tile w = tile_at<PAIR>(a, start, t, g);
      const int acc = i & 1;
      if (!zero &&
          !tc::wait_warp(smem_u32(&acc_full[acc]), uint32_t(i >> 1) & 1, abort_flag, a.status))
        break;
      tc::fence_after();
      const int r0 = int(rank) * 128 + q * 32;     // this warp's first row of the tile
      const uint32_t taddr = tmem + (uint32_t(q * 32) << 16) + uint32_t(acc ? a.acc1 : 0);
      uint8_t* out = static_cast<uint8_t*>(a.d) + (int64_t(w.row0 + r0) * a.stride + w.col0) * es;
#pragma unroll 1
      for (int k = 0; k < halves; ++k) {
        // columns shared with the other sum first: the last of sum 0, the
        // first of sum 1
        const int c0 = (acc ? k : halves - 1 - k) * 128;
        uint32_t v[4][32];
        if (!zero) {
#pragma unroll
          for (int j = 0; j < 4; ++j) tc::tmem_ld32(taddr + c0 + j * 32, v[j]);
          tc::tmem_wait_ld();
          if (k == (shared_cols ? 0 : halves - 1)) {
            // hand the columns to the MMA warp: for the other sum's next
            // tile, or for this sum's.  (The loads are complete; a release
            // would also wait for this warp's stores to D.)
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
              const uint32_t bar = smem_u32(&acc_empty[shared_cols ? acc ^ 1 : acc]);
              if (PAIR && rank != 0)
                tc::arrive_cluster_relaxed(tc::map_to_rank(bar, 0));
              else
                mbar_arrive(bar);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 32; ++e) v[j][e] = 0u;
        }
        // 32 rows x 128 bytes at a time through a staging buffer: 64 columns
        // of bf16 or 32 of fp32, 16-byte pieces rotated by row as the 128-byte
        // swizzle has them
#pragma unroll
        for (int j = 0; j < 4; j += BF16 ? 2 : 1) {
          const int col = c0 + j * 32;             // first column of these 128 bytes
          if (col >= a.bn || w.col0 + col >= a.N) continue;   // (uniform)
          const uint32_t buf = staging + (turn & 1) * (32 * 128);
          ++turn;
          if (lane == 0) bulk_wait_read<1>();      // the store that last read this buffer
          __syncwarp();
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            uint32_t x[4];
            if constexpr (BF16) {
              const uint32_t* s = p < 4 ? &v[j][p * 8] : &v[j + 1][(p - 4) * 8];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                x[e] = pack_bf16x2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = v[j][p * 4 + e];
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             buf + lane * 128 + ((p ^ (lane & 7)) << 4)),
                         "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
                         : "memory");
          }
          constexpr int kWide = BF16 ? 64 : 32;
          if (a.vec && r0 + 32 <= w.rows && w.col0 + col + kWide <= a.n_copied) {
            // one copy for the 32 rows
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              tensor_store_2d(&a.map_d, buf, w.col0 + col, w.row0 + r0);
              bulk_commit();
            }
          } else {
            // rows that end with the range, or rows of D that no copy can address
            __syncwarp();
            store_rows<BF16>(buf, out + int64_t(col) * es, a.stride * es, min(32, w.rows - r0),
                             min(min(a.N - w.col0, a.bn) - col, kWide));
            __syncwarp();
            if (lane == 0) bulk_commit();   // an empty group: the buffers' turns count groups
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();   // this warp's copies to D have been written
  }

  // ------------------------------------------------------------ teardown
  __syncthreads();
  if (warp == 1) {
    // every MMA has completed before the tensor memory is released
    if (lane == 0) {
      if (rank == 0) tc::commit<PAIR>(smem_u32(drain));
      tc::wait_drain(smem_u32(drain), 0);
    }
    __syncwarp();
  }
  tc::fence_before();
  if constexpr (PAIR) tc::cluster_sync();   // neither CTA leaves while the pair still works
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc<PAIR>(tmem, 512);
  }
}

template <bool PAIR, bool BF16>
fo_status launch(const GemmArgs& a, int grid, cudaStream_t st) {
  static std::once_flag once[64];
  static cudaError_t err[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FO_ERR_CUDA;
  const int slot = dev < 64 ? dev : 63;
  std::call_once(once[slot], [&] {
    err[slot] = cudaFuncSetAttribute(mx_gemm_kernel<PAIR, BF16>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  });
  if (err[slot] != cudaSuccess) return FO_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = PAIR ? 2 : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, mx_gemm_kernel<PAIR, BF16>, a) != cudaSuccess) {
    cudaGetLastError();
    return FO_ERR_CUDA;
  }
  return FO_OK;
}

}  // namespace

fo_status launch_mx_gemm(int64_t M, int64_t N, int64_t K, const void* a_codes,
                         const void* a_scales, const void* b_codes, const void* b_scales,
                         int32_t n_groups, const int32_t* group_first,
                         const int32_t* group_rows, void* D, fo_type type, int64_t row_stride,
                         int32_t* dev_status, void* stream) {
  if (M == 0 || N == 0) return FO_OK;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FO_ERR_CUDA;
  const int64_t groups = n_groups > 0 ? n_groups : 1;
  const int64_t kb = mx_up(K, 128) / 128;               // blocks of scales per row of blocks
  const int64_t mb = mx_up(M, 128) / 128, nb = mx_up(N, 128) / 128 * groups;
  // A pair reads half as much of B per CTA, and its tiles are four times as
  // large: while those of one CTA all run at once, they are faster (512 x 4096 x
  // 4096: 10.4 us, pairs 12.4; 1024 x 4096 x 4096: 14.5 and 12.4), and with no
  // more rows than one CTA takes a pair's second half would be empty.
  // So it is with experts of 128 rows or less on average, whose rounded rows A has
  // (16 experts of 2 rows, N = 9123, K = 877: 25 us, pairs 37).
  const bool pair = M > 128 && mb >= 2 * groups && mb * (nb / groups) > sms;
  GemmArgs a{};
  a.bn = pair ? 256 : 128;
  a.acc1 = kSf0 - a.bn < a.bn ? kSf0 - a.bn : a.bn;
  if (K > 0) {
    const uint64_t pitch = uint64_t(kb) * 64;
    const uint32_t b_rows = uint32_t(pair ? a.bn / 2 : a.bn);
    if (!encode_tensor_map(&a.map_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, a_codes, pitch, mb * 128, pitch,
                           128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tensor_map(&a.map_b, CU_TENSOR_MAP_DATA_TYPE_UINT8, b_codes, pitch, nb * 128, pitch,
                           128, b_rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tensor_map(&a.map_sa, CU_TENSOR_MAP_DATA_TYPE_UINT32, a_scales, kb * 128, mb,
                           kb * 512, 256, 1, CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !encode_tensor_map(&a.map_sb, CU_TENSOR_MAP_DATA_TYPE_UINT32, b_scales, kb * 128, nb,
                           kb * 512, 256, kSbBlocks, CU_TENSOR_MAP_SWIZZLE_NONE))
      return FO_ERR_CUDA;
  }
  a.first = group_first;
  a.rows = group_rows;
  a.d = D;
  a.stride = row_stride;
  a.M = int32_t(M);
  a.N = int32_t(N);
  a.n_pad = int32_t(mx_up(N, 128));
  a.n_groups = int32_t(groups);
  a.grouped = n_groups > 0;
  a.k_stages = int32_t((K + kStageCols - 1) / kStageCols);
  a.k_steps = int32_t((K + 63) / 64);
  const bool bf16 = type == FO_TYPE_BF16;
  const int es = bf16 ? 2 : 4;
  a.vec = ((reinterpret_cast<uintptr_t>(D) | uintptr_t(row_stride) * es) & 15) == 0 &&
          row_stride * es < (int64_t(1) << 40);
  // A copy leaves out whole 16-byte pieces past N, not single elements: the
  // last columns are copied only if N ends on such a piece.
  a.n_copied = (N * es) % 16 == 0 ? int32_t(mx_up(N, 64)) : int32_t(N);
  if (a.vec && !encode_tensor_map(&a.map_d,
                                  bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                                  D, N, M, uint64_t(row_stride) * es, 128 / es, 32,
                                  CU_TENSOR_MAP_SWIZZLE_128B))
    return FO_ERR_CUDA;
  a.status = dev_status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // no more workers than tiles (with experts: than any ranges can make)
  const int64_t most = (mb + groups) * ((N + a.bn - 1) / a.bn);
  const int64_t workers = pair ? sms / 2 : sms;
  const int64_t use = most < workers ? most : workers;
  if (pair) return bf16 ? launch<true, true>(a, int(2 * use), st) : launch<true, false>(a, int(2 * use), st);
  return bf16 ? launch<false, true>(a, int(use), st) : launch<false, false>(a, int(use), st);
}

}  // namespace fo
