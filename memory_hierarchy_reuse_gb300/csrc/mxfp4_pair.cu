// The 4-bit product for many rows: persistent CTA pairs (tcgen05 cta_group::2)
// on tiles of 256 rows x 256 (or fewer) columns of C, K in stages of 256.
//
// Bound by the tensor pipe, and next to it by shared memory: a 256 x 256 x 64
// MMA takes 128 cycles, in which an SM reads 128 rows of A and of B (32 bytes
// each, 8 KB) and TMA writes as much for the stages ahead: 128 bytes a cycle,
// all that shared memory moves.  So both operands are staged once a pair (each
// CTA holds its 128 rows of A and half of B), and nothing else but the scales
// (1/16 of the operands, through tcgen05.cp) touches shared memory in the main
// loop.  GB300, call after call on the same operands: 8192^3 in 149 us, 7.4 PFLOP/s (a
// stage at 7.7, the rest is the last round and the ends), 4096^3 in 26.2 (29.3 on other
// operands every call, which come from HBM); 333 x 5000 x 4104 in 11.2, most of it the 17
// stages' and the launch's latency.
//
// TMEM: two accumulators of 256 columns and two sets of scales (24 columns
// each: A's 128 rows and B's 256 rows x 8 blocks) would take 560 of the 512
// columns.  The accumulators overlap by 48: the epilogue drains the columns
// that the other one needs first, and the next tile's MMAs start while it
// drains the rest.  A last round that leaves half of the pairs idle is done as
// halves of 128 columns.  Narrower tiles have both accumulators side by side; tiles of
// 192 columns start in the middle of a scale tile every other time, and address
// B's scales from there on (64 rows are two TMEM columns; widths that would
// start at an odd column are not used).
#include <cstdio>
#include <type_traits>

#include "mhr_gemm.h"
#include "mhr_mxfp4.h"
#include "mxfp4_common.cuh"

namespace mhr {
namespace mx {
namespace {

constexpr int TILE_M = 256;                  // rows of a pair's tile
constexpr int MAX_BN = 256;                  // its columns: 256, 192 or 128
constexpr int HALF = 128;
constexpr int BK_BYTES = 128;                // 256 columns of K a stage: one swizzle row
constexpr int OP_BYTES = HALF * BK_BYTES;    // this CTA's A rows, and its half of B at most
constexpr int OFF_B = OP_BYTES;
constexpr int OFF_SFA = 2 * OP_BYTES;        // 2 scale tiles: 128 rows x 8 blocks
constexpr int OFF_SFB = OFF_SFA + 1024;      // up to 2 x 2: all columns of the tile
constexpr int STAGE_BYTES = OFF_SFB + 2048;  // 35 KB
constexpr int STAGES = 5;
constexpr int EPI_WARPS = 4;
constexpr int EPI_BUF = 32 * 128;            // 32 rows of 128 bytes
constexpr int EPI_OFF = STAGES * STAGE_BYTES;
constexpr int SMEM = EPI_OFF + EPI_WARPS * 2 * EPI_BUF + 1024;
constexpr int THREADS = 192;
constexpr uint32_t OVERLAP = 48;             // columns that two accumulators of 256 share
constexpr uint32_t TMEM_COLS = 512;

// 128-row scale tiles of B that a tile of bn columns brings (192 rows that start
// 64 into one end with the second).
__host__ __device__ constexpr int sf_tiles(int bn) { return (bn + 127) / 128; }

struct PairParams {
  int32_t M, N;
  int32_t tiles_m, tiles_n, num_kb;
  int32_t group;           // tile rows walked together, column by column
  int32_t whole, units;    // units of work: tiles done whole, then halves (128 columns) of the rest
  int32_t blocks;
  void* C;
  int64_t ldc;
  int32_t c_dtype;
  uint32_t* status;
  uint64_t wait_limit_ns;
  int32_t inject_stall;
};

__device__ __forceinline__ void tile_at(int t, const PairParams& p, int& tm, int& tn) {
  const int group_size = p.group * p.tiles_n;
  const int g = t / group_size, first = g * p.group;
  const int gm = min(p.tiles_m - first, p.group), r = t - g * group_size;
  tm = first + r % gm;
  tn = r / gm;
}

// First column of unit u, and its tile row.  Halves are of tiles of 256 columns.
__device__ __forceinline__ int unit_at(int u, int bn, const PairParams& p, int& tm) {
  int tn;
  const int half = u < p.whole ? 0 : (u - p.whole) & 1;
  tile_at(u < p.whole ? u : p.whole + ((u - p.whole) >> 1), p, tm, tn);
  return tn * bn + half * 128;
}

__device__ __forceinline__ uint32_t pack16(int c_dtype, uint32_t lo, uint32_t hi) {
  const float a = __uint_as_float(lo), b = __uint_as_float(hi);
  if (c_dtype == MHR_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Warp roles, barriers and the way a timeout unwinds are those of the bf16
// and tf32 pair kernel (tc_gemm_pair.cu): warp 0 producer, warp 1 MMA issuer
// (rank 0), warps 2-5 epilogue; full[s] and released[b] in rank 0, empty[s]
// and acc_full[b] in both CTAs.  released[b]: accumulator b -- of two that
// overlap, the columns that the other one shares -- has been read by all 8
// epilogue warps.
// WIDE: C is fp32, else 16 bits.  TMA_STORE: C goes out by TMA.
template <int BN, bool WIDE, bool TMA_STORE>
__global__ void __launch_bounds__(THREADS, 1)
    mxfp4_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmBHalf,
                      const __grid_constant__ CUtensorMap tmSA,
                      const __grid_constant__ CUtensorMap tmSB,
                      const __grid_constant__ CUtensorMap tmC, const PairParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ alignas(8) uint64_t bars[2 * STAGES + 6];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ volatile uint32_t peer_loaded;  // rank 0: stages that rank 1 loaded
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem), bar0 = smem_u32(bars);
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (STAGES + s); };
  auto acc_bar = [&](uint32_t b) { return bar0 + 8u * (2 * STAGES + b); };
  auto released_bar = [&](uint32_t b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);
  const uint32_t peer_done_bar = bar0 + 8u * (2 * STAGES + 5);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  constexpr bool overlap = BN == MAX_BN;
  constexpr uint32_t acc1 = overlap ? MAX_BN - OVERLAP : BN;  // the second accumulator
  constexpr int SF_TILES = sf_tiles(BN);
  constexpr uint32_t sf_set = 8 + 8 * SF_TILES;               // columns of a set of scales
  constexpr uint32_t SF_SETS = overlap ? 2 : STAGES;
  static_assert(acc1 + BN + SF_SETS * sf_set <= TMEM_COLS, "TMEM");
  static_assert(!overlap || 128 + STAGES * 16 <= acc1, "a half and its scales");
  constexpr uint32_t stage_tx = OP_BYTES + BN / 2 * BK_BYTES + 1024 * (1 + SF_TILES);
  constexpr uint32_t half_tx = stage_tx - (BN / 2 - 64) * BK_BYTES;
  const uint32_t peer_abort = mapa_shared(smem_u32(const_cast<int*>(&abort_flag)), rank ^ 1u);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_bar(b), 1);
      mbar_init(released_bar(b), 2 * EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    mbar_init(peer_done_bar, 1);
    abort_flag = 0;
    peer_loaded = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
    if (TMA_STORE) tma_prefetch_desc(&tmC);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint64_t limit = p.wait_limit_ns;
  // (No grid_launch_dependents(): a quantisation let in early, call after call, cost
  // more -- 8192^3 with its quantisation 195 us against 186, 333 x 5000 x 4104 13.9
  // / 13.6 -- than a product let in early gains: 10.7 / 11.0 us for the latter.)
  grid_dependency_wait();

  auto give_up = [&](uint32_t bit) {  // by one thread: both CTAs unwind
    if (!abort_flag) atomicOr(p.status, bit);
    abort_flag = 1;
    st_shared_cluster_u32(peer_abort, 1u);
  };

  if (warp == 0) {
    uint32_t it = 0, s = 0, ph = 1;  // stages armed and loaded; ring position, phase to wait for
    const bool stall = p.inject_stall && blockIdx.x == 0;  // test hook: stage 0 never fills
    const uint32_t fb0 = mapa_shared(full_bar(0), 0);
    bool ok = true;
    auto load_unit = [&](auto half, int u) {
      constexpr bool HALF_UNIT = decltype(half)::value;
      constexpr uint32_t tx = HALF_UNIT ? half_tx : stage_tx;
      int tm;
      const int n0 = unit_at(u, BN, p, tm);
      const int m0 = tm * TILE_M + static_cast<int>(rank) * HALF;
      const int nb0 = n0 + static_cast<int>(rank) * (HALF_UNIT ? 64 : BN / 2);
      for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
        if (!__all_sync(0xffffffffu,
                        mbar_wait_bounded(empty_bar(s), ph, limit, &abort_flag))) {
          if (lane == 0) give_up(kErrTimeoutProducer);
          ok = false;
          break;
        }
        const uint32_t st = sbase + s * STAGE_BYTES, fb = fb0 + 8u * s;
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * tx);
          if (!(stall && it == 0)) {
            tma_load_2d_pair(st, &tmA, fb, kb * BK_BYTES, m0);
            tma_load_2d_pair(st + OFF_B, HALF_UNIT ? &tmBHalf : &tmB, fb, kb * BK_BYTES, nb0);
            // (boxes past the last row or block are filled with zeros)
            tma_load_3d_pair(st + OFF_SFA, &tmSA, fb, 0, 2 * kb, m0 / 128);
            tma_load_3d_pair(st + OFF_SFB, &tmSB, fb, 0, 2 * kb, n0 / 128);
          }
        }
        __syncwarp();
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
    };
    int u = cluster;
    for (; ok && u < p.whole; u += clusters) load_unit(std::false_type{}, u);
    if constexpr (BN == MAX_BN)
      if (ok && u < p.units) load_unit(std::true_type{}, u);
    if (lane == 0) {
      // Both CTAs' loads complete in rank 0, which waits for all of them --
      // counting as done what either side never issued -- before either CTA
      // may leave.
      volatile int never = 0;
      if (!leader) {
        st_shared_cluster_u32(
            mapa_shared(smem_u32(const_cast<uint32_t*>(&peer_loaded)), 0), it);
        mbar_arrive_cluster(mapa_shared(peer_done_bar, 0));
      } else {
        uint32_t it1 = it;
        if (mbar_wait_bounded<true>(peer_done_bar, 0, 2 * limit, &never))
          it1 = peer_loaded;
        else
          atomicOr(p.status, kErrTimeoutDrain);
        const uint32_t hi = it > it1 ? it : it1;
        const uint32_t whole_stages =
            cluster < p.whole ? ((p.whole - 1 - cluster) / clusters + 1) * p.num_kb : 0;
        for (uint32_t i = hi > STAGES ? hi - STAGES : 0; i < hi; ++i) {
          const uint32_t s = i % STAGES, ph = (i / STAGES) & 1u;
          const bool armed = i < it, loaded0 = armed && !(stall && i == 0), loaded1 = i < it1;
          const uint32_t tx = i < whole_stages ? stage_tx : half_tx;
          if (!armed) {
            mbar_arrive_expect_tx(full_bar(s), tx);
          } else {
            const uint32_t missing = (loaded0 ? 0u : tx) + (loaded1 ? 0u : tx);
            if (missing) {  // once the MMA issuer has given up on the stage
              mbar_wait_bounded(full_bar(s), ph, 2 * limit, &abort_flag);
              mbar_complete_tx(full_bar(s), missing);
            }
          }
          if (!mbar_wait_bounded(full_bar(s), ph, limit, &never))
            atomicOr(p.status, kErrTimeoutDrain);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader) {
      const int tail = (p.blocks - (p.num_kb - 1) * 8 + 1) / 2;  // MMAs of a tile's last stage
      uint32_t it = 0, t = 0, s = 0, ph = 0;       // stages done; ring position and its phase
      uint32_t s2 = STAGES - 2, ph2 = 1;           // the same two stages back
      bool ok = true;
      // a warp-uniform outcome: every lane polls
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, limit, &abort_flag)) != 0;
      };
      auto multiply_unit = [&](auto half, int u) {
        constexpr bool HALF_UNIT = decltype(half)::value;
        constexpr int COLS = HALF_UNIT ? 128 : BN, TILES = HALF_UNIT ? 1 : SF_TILES;
        constexpr uint32_t sf_k = 4 * TILES;  // columns of B's scales for 128 columns of K
        const uint32_t id0 = make_idesc_mxf4(TILE_M, COLS, 0);
        const uint32_t id2 = make_idesc_mxf4(TILE_M, COLS, 2);
        // this accumulator's last tile but one has been read; of two that
        // overlap, the other one's shared columns (and with them, by the same
        // warps earlier, all of this one)
        const uint32_t before = overlap ? t - 1 : t - 2;
        if (t >= (overlap ? 1u : 2u) &&
            !wait(released_bar(before & 1u), (before >> 1) & 1u)) {
          if (lane == 0) give_up(kErrTimeoutMma);
          ok = false;
          return;
        }
        tc_fence_after();
        const uint32_t d = tmem + (t & 1u ? acc1 : 0);
        uint32_t sf_row = 0;  // TMEM column of the tile's first row in its scale tile
        if constexpr (BN % 128 != 0) {
          int tm;
          sf_row = (unit_at(u, BN, p, tm) & 127) >> 5;
        }
        for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
          // A stage's scales have columns of their own -- whoever read them last
          // had finished before the stage was filled again -- or alternate
          // between two sets: then the MMAs two stages back, the last to read
          // this one, have to have finished.  (Both barriers polled once
          // together; mostly that is all.)
          const bool older = !HALF_UNIT && SF_SETS < STAGES && it >= 2;
          bool there = mbar_try_wait(full_bar(s), ph);
          there = (!older || mbar_try_wait(empty_bar(s2), ph2)) && there;
          if (!__all_sync(0xffffffffu, there) &&
              ((older && !wait(empty_bar(s2), ph2)) || !wait(full_bar(s), ph))) {
            if (lane == 0) give_up(kErrTimeoutMma);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = sbase + s * STAGE_BYTES;
          const uint32_t a = desc_lo(st), bb = a + (OFF_B >> 4);
          const uint32_t ca = a + (OFF_SFA >> 4), cb = a + (OFF_SFB >> 4);
          // (a half's are next to it: the columns that its accumulator leaves free)
          const uint32_t sfa = HALF_UNIT ? d + 128 + s * 16
                                         : tmem + acc1 + BN +
                                               (SF_SETS < STAGES ? it & 1u : s) * sf_set;
          const uint32_t sfb = sfa + 8;
          const uint32_t first = kb > 0 ? 1u : 0u;
          const bool full = kb + 1 < p.num_kb || tail == 4;
          if (elect_one()) {
            // columns: A's tiles 0 and 1 of K; B's for tile 0 of K, then for tile 1
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              copy_scale_tile<2>(sfa + 4 * i, ca + 32 * i);
              #pragma unroll
              for (int j = 0; j < TILES; ++j)
                copy_scale_tile<2>(sfb + sf_k * i + 4 * j, cb + 64 * j + 32 * i);
            }
            const uint32_t sb = sfb + sf_row;
            if (full) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_mxf4<2>(d, a + 2 * kk, bb + 2 * kk, kk & 1 ? id2 : id0, sfa + 4 * (kk >> 1),
                            sb + sf_k * (kk >> 1), kk > 0 ? 1u : first);
            } else {
              for (int kk = 0; kk < tail; ++kk)
                mma_mxf4<2>(d, a + 2 * kk, bb + 2 * kk, kk & 1 ? id2 : id0, sfa + 4 * (kk >> 1),
                            sb + sf_k * (kk >> 1), kk > 0 ? 1u : first);
            }
            mma_commit_pair_multicast(empty_bar(s), 0x3);
            if (kb + 1 == p.num_kb) mma_commit_pair_multicast(acc_bar(t & 1u), 0x3);
          }
          __syncwarp();
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
          if (++s2 == STAGES) {
            s2 = 0;
            ph2 ^= 1u;
          }
        }
      };
      int u = cluster;
      for (; ok && u < p.whole; u += clusters, ++t) multiply_unit(std::false_type{}, u);
      if constexpr (BN == MAX_BN)
        if (ok && u < p.units) multiply_unit(std::true_type{}, u);
      if (elect_one()) mma_commit_pair(drain_bar);
      __syncwarp();
      volatile int never = 0;
      if (!mbar_wait_bounded(drain_bar, 0, limit, &never) && lane == 0)
        atomicOr(p.status, kErrTimeoutDrain);
    }
    __syncwarp();
  } else {
    const int q = warp & 3, ew = warp - 2;
    constexpr int COLS = WIDE ? 32 : 64;       // columns of a piece: 128 bytes a row
    constexpr int FIRST = WIDE ? 2 : 1;        // pieces that hold the overlapping columns
    constexpr int pieces = BN / COLS;
    constexpr int release = overlap ? FIRST - 1 : pieces - 1;  // the piece that frees the accumulator
    uint32_t t = 0, chunk = 0;
    for (int u = cluster; u < p.units; u += clusters, ++t) {
      const uint32_t b = t & 1u;
      if (!__all_sync(0xffffffffu,
                      mbar_wait_bounded(acc_bar(b), (t >> 1) & 1u, limit, &abort_flag, 128))) {
        if (lane == 0) give_up(kErrTimeoutEpilogue);
        __syncwarp();
        break;
      }
      tc_fence_after();
      int tm;
      const int n0 = unit_at(u, BN, p, tm);
      const int row0 = tm * TILE_M + static_cast<int>(rank) * HALF + q * 32;
      const bool half = u >= p.whole;  // (the cluster's last unit)
      const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + (b ? acc1 : 0);
#pragma unroll 1
      for (int i = 0; i < (half ? 128 / COLS : pieces); ++i) {
        // of two that overlap, the first accumulator's shared columns are its
        // last, the second's its first
        const int c = b || half || !overlap ? i : (i < FIRST ? pieces - FIRST + i : i - FIRST);
        uint32_t r[32];
        tmem_ld_32cols(taddr + c * COLS, r);
        if constexpr (!WIDE) {
          uint32_t r2[32];
          tmem_ld_32cols(taddr + c * COLS + 32, r2);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) r[j] = pack16(p.c_dtype, r[2 * j], r[2 * j + 1]);
#pragma unroll
          for (int j = 0; j < 16; ++j) r[16 + j] = pack16(p.c_dtype, r2[2 * j], r2[2 * j + 1]);
        } else {
          tmem_ld_wait();
        }
        if (i == release) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(released_bar(b), 0));
        }
        // One row a lane into a 128-byte swizzled box (conflict-free), then
        // out by TMA, or a row at a time where C is not aligned for it.
        const uint32_t stg = sbase + EPI_OFF + (ew * 2 + (chunk & 1u)) * EPI_BUF;
        ++chunk;
        if (TMA_STORE) {
          if (lane == 0) bulk_wait_group_read<1>();
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t at = stg + lane * 128 + ((j ^ (lane & 7)) << 4);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(r[4 * j]),
                       "r"(r[4 * j + 1]), "r"(r[4 * j + 2]), "r"(r[4 * j + 3])
                       : "memory");
        }
        const int col0 = n0 + c * COLS;
        if constexpr (TMA_STORE) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmC, stg, col0, row0);
            bulk_commit_group();
          }
        } else {
          __syncwarp();
          const int rows = min(32, p.M - row0);
          for (int rr = 0; rr < rows; ++rr) {
            uint32_t v;
            asm volatile("ld.shared.b32 %0, [%1];"
                         : "=r"(v)
                         : "r"(stg + rr * 128 + (((lane >> 2) ^ (rr & 7)) << 4) + (lane & 3) * 4)
                         : "memory");
            const int64_t row = static_cast<int64_t>(row0 + rr) * p.ldc;
            if constexpr (WIDE) {
              if (col0 + lane < p.N) static_cast<uint32_t*>(p.C)[row + col0 + lane] = v;
            } else {
              uint16_t* dst = static_cast<uint16_t*>(p.C) + row + col0 + 2 * lane;
              const int left = p.N - (col0 + 2 * lane);
              if (left >= 2 && (reinterpret_cast<uintptr_t>(dst) & 3u) == 0) {
                *reinterpret_cast<uint32_t*>(dst) = v;
              } else {
                if (left >= 1) dst[0] = static_cast<uint16_t>(v);
                if (left >= 2) dst[1] = static_cast<uint16_t>(v >> 16);
              }
            }
          }
          __syncwarp();
        }
      }
    }
    if (TMA_STORE) {
      if (lane == 0) bulk_wait_group<0>();
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the pair's MMAs or arrivals may touch it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

// Tiles of the last round that are done as two halves of 128 columns each, by two
// clusters: all of them where that many are free, of tiles of 256 columns.  GB300,
// with halves and without: 4096^3 (28 tiles left of 256) 26.8 / 28.1 us, 8192^3 (36
// of 1024) 155.1 / 157.2.
int64_t halves(int bn, int64_t tiles, int clusters) {
  const int64_t rest = tiles % clusters;
  return bn == MAX_BN && 2 * rest <= clusters ? rest : 0;
}

// One launch on as many clusters as can run at once (at most one a unit).
template <int BN, bool WIDE, bool TMA_STORE>
cudaError_t launch_t(const CUtensorMap (&m)[6], PairParams p, int device,
                     cudaLaunchConfig_t cfg) {
  auto kern = mxfp4_pair_kernel<BN, WIDE, TMA_STORE>;
  static int most[64];  // by device; under the library's lock
  int clusters = device < 64 ? most[device] : 0;
  if (!clusters) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    if ((e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg)) != cudaSuccess) return e;
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    if (device < 64) most[device] = clusters;
  }
  const int rest = static_cast<int>(halves(BN, p.whole, clusters));
  p.units = p.whole + rest;
  p.whole -= rest;
  if (p.units < clusters) clusters = p.units;
  cfg.gridDim = dim3(2 * clusters);
  cfg.numAttrs = 2;
  char name[48];
  snprintf(name, sizeof(name), "mxfp4_pair_kernel<n%d>", BN);
  note_main_kernel(name, 2 * clusters, p.units);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, m[0], m[1], m[2], m[3], m[4], m[5], p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int BN>
cudaError_t launch_bn(const CUtensorMap (&m)[6], const PairParams& p, bool wide, bool c_tma,
                      int device, const cudaLaunchConfig_t& cfg) {
  if (wide)
    return c_tma ? launch_t<BN, true, true>(m, p, device, cfg)
                 : launch_t<BN, true, false>(m, p, device, cfg);
  return c_tma ? launch_t<BN, false, true>(m, p, device, cfg)
               : launch_t<BN, false, false>(m, p, device, cfg);
}

// Scales as 512-byte tiles: tile_rows x kt of them, boxes of 2 x `rows`.
bool scale_map(CUtensorMap* map, const uint8_t* scales, int64_t rows, int64_t kt, uint32_t box) {
  const uint64_t dims[3] = {128, static_cast<uint64_t>(kt), static_cast<uint64_t>((rows + 127) / 128)};
  const uint64_t pitch[2] = {512, static_cast<uint64_t>(kt) * 512};
  const uint32_t boxes[3] = {128, 2, box};
  return encode_tmap_3d(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, scales, dims, pitch, boxes) ==
         CUDA_SUCCESS;
}

}  // namespace

// Tile columns.  The time is that of the busiest cluster: its rounds of tiles of
// num_kb stages each, a last round of halves, and the last tile's epilogue, in
// units of 0.72 ns.  GB300: a stage of 256 / 192 / 128 columns takes 470 / 376 /
// 345 of them with all clusters at work, one of a half 414 (4096^3 in 26.4 / 26.6 /
// 32.2 us, 8192^3 in 149.7 / 155.4 / 202.5).  Narrower tiles put more clusters to
// work on few tiles (2000 x 300 x 4000: 11.6 us with 128 columns, 14.0 with 192; 6144
// x 4096 x 4096: 36.0 with 192, 38.2 with 256), wider ones load less.
int plan_pair_bn(int64_t M, int64_t N, int64_t K, int clusters, double* best_t) {
  const int64_t stages = (scale_tiles(K) + 1) / 2;
  int best = MAX_BN;
  for (int bn = MAX_BN; bn >= 128; bn -= 64) {
    const double stage = bn == 256 ? 470 : bn == 192 ? 376 : 345;
    const int64_t tiles = (M + TILE_M - 1) / TILE_M * ((N + bn - 1) / bn);
    const int64_t rest = halves(bn, tiles, clusters);
    const int64_t rounds = (tiles - rest + clusters - 1) / clusters;
    const double t = static_cast<double>(stages) * (rounds * stage + (rest ? 414 : 0)) +
                     6.0 * (rest ? 128 : bn);
    if (bn == MAX_BN || t < *best_t) {
      *best_t = t;
      best = bn;
    }
  }
  return best;
}

double pair_time(int64_t M, int64_t N, int64_t K, int clusters) {
  double t = 0;
  plan_pair_bn(M, N, K, clusters, &t);
  return 4.1 + 0.72e-3 * t;
}

cudaError_t launch_pair(const ProductArgs& a, const DeviceCtl& ctl, cudaStream_t s) {
  const bool wide = a.c_dtype == MHR_F32;
  const int64_t size = wide ? 4 : 2;
  // TMA stores clip a box at C's inner extent in 16-byte units only
  const bool c_tma = reinterpret_cast<uintptr_t>(a.C) % 16 == 0 && a.ldc * size % 16 == 0 &&
                     a.N * size % 16 == 0;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(2 * (ctl.sm_count / 2));
  int device = 0;
  if (const cudaError_t e = cudaGetDevice(&device); e != cudaSuccess) return e;

  PairParams p;
  p.M = static_cast<int32_t>(a.M);
  p.N = static_cast<int32_t>(a.N);
  // (gemm_testing_set_pair_tile_n forces a width, rounded to one that exists)
  double t;
  const int bn = ctl.pair_tile_n ? ctl.pair_tile_n / 64 * 64
                                 : plan_pair_bn(a.M, a.N, a.K, ctl.sm_count / 2, &t);
  p.tiles_m = static_cast<int32_t>((a.M + TILE_M - 1) / TILE_M);
  p.tiles_n = static_cast<int32_t>((a.N + bn - 1) / bn);
  const int64_t kt = scale_tiles(a.K);
  p.num_kb = static_cast<int32_t>((kt + 1) / 2);
  // The order of the tiles, for L2: whole columns of up to 32 tiles; two rows at a
  // time of a tall C; rows where K is short, and C's stores, in longer runs along a
  // row, are much of the traffic.  GB300, groups of 32 / 8 / 2 / 1 rows: 8192^3 150.7
  // / 155.5 / 152.9 / 153.4 us, 8192 x 16384 x 4096 169.0 / 181.2 / 177.5 / 175.7;
  // 32768 x 4096 x 4096 173.5 / 168.8 / 167.8 for the first three; 7000 x 9000 x 3000
  // 80.8 / 78.8 / 77.0 / 77.2, 16384 x 16384 x 2048 220.8 / 238.8 / 228.6 / 212.3.
  p.group = p.tiles_m > 32 && p.tiles_n <= 32 ? 2 : p.num_kb < 16 ? 1 : 32;
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  if (tiles > 0x3fffffff) return cudaErrorInvalidConfiguration;
  p.whole = static_cast<int32_t>(tiles);  // (launch_t takes off those that are halved)
  p.blocks = static_cast<int32_t>(blocks_of(a.K));
  p.C = a.C;
  p.ldc = a.ldc;
  p.c_dtype = a.c_dtype;
  p.status = ctl.status;
  p.wait_limit_ns = ctl.wait_limit_ns;
  p.inject_stall = ctl.inject_stall;
  const int64_t row_bytes = static_cast<int64_t>(p.blocks) * 16;
  CUtensorMap m[6];
  if (encode_tmap_2d(&m[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, a.A, row_bytes, a.M, a.lda, BK_BYTES,
                     HALF, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
      encode_tmap_2d(&m[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, a.B, row_bytes, a.N, a.ldb, BK_BYTES,
                     bn / 2, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
      encode_tmap_2d(&m[2], CU_TENSOR_MAP_DATA_TYPE_UINT8, a.B, row_bytes, a.N, a.ldb, BK_BYTES,
                     64, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
      !scale_map(&m[3], a.sfa, a.M, kt, 1) || !scale_map(&m[4], a.sfb, a.N, kt, sf_tiles(bn)))
    return cudaErrorInvalidValue;
  m[5] = m[0];
  if (c_tma && encode_tmap_2d(&m[5],
                              wide ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                              a.C, a.N, a.M, a.ldc * size, 128 / size, 32,
                              CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  if (bn == 256) return launch_bn<256>(m, p, wide, c_tma, device, cfg);
  if (bn == 192) return launch_bn<192>(m, p, wide, c_tma, device, cfg);
  return launch_bn<128>(m, p, wide, c_tma, device, cfg);
}

}  // namespace mx
}  // namespace mhr
