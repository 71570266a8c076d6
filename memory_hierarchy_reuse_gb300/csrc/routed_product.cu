// The experts' products (gemm_routed_product) and their weights' gradient
// (gemm_routed_weight_grad): persistent CTA pairs (tcgen05 cta_group::2).
//
// A pair's tile has the output's columns -- features -- on the MMA's rows, 256 of
// them, and rows of tokens (or, of a gradient, of features of x) on its columns, 32
// to 256: an expert's rows are few and of any number, its features many, so the side
// that varies is the one whose length an MMA takes in steps.  The transposed result
// costs nothing: a lane of TMEM is a feature, so a warp's store of one row is 32
// neighbours.  Which tiles there are stands in the offsets on the device alone; every
// CTA sums them up in shared memory and takes every clusters-th.
//
// Operands:          features side               rows side
//   product           W_e (K x N): MN-major       x rows, K-major
//   transposed        W_e (N x K): K-major        x rows, K-major
//   weight gradient   gradient rows, MN-major     x rows, MN-major
// Rows that an index picks come by TMA's gather of four rows, a lane four rows; a row
// outside its matrix -- past an expert's last, or an index out of range -- is zeros.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdio>

#include "mhr_gemm.h"
#include "mhr_mxfp4.h"
#include "mxfp4_common.cuh"
#include "routed_internal.h"

namespace mhr {
namespace routed {
namespace {

using mx::elect_one;
using mx::tma_load_3d_pair;

constexpr uint32_t ALL = 0xffffffffu;
constexpr int TILE_F = 256;                  // features of a pair's tile
constexpr int HALF = 128;
constexpr int MAX_ROWS = 256;                // rows of a pair's tile
constexpr int BK = 64;                       // of the sum a stage: one swizzle row of 128 bytes
constexpr int A_BYTES = HALF * BK * 2;       // this CTA's features
constexpr int BOX = 64 * 128;                // 64 rows of 128 bytes
constexpr int B_BYTES = HALF * BK * 2;       // this CTA's half of the rows, at most
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;  // 32 KB
constexpr int STAGES = 6;
constexpr int EPI_WARPS = 4;
constexpr int THREADS = 192;
constexpr int SMEM = STAGES * STAGE_BYTES + 1024;
constexpr uint32_t TMEM_COLS = 2 * MAX_ROWS;

enum Mode { PRODUCT = 0, TRANSPOSED = 1, GRADIENT = 2 };

struct Params {
  const int32_t* offsets;
  const int32_t* gather;   // rows of x over `top`, or null
  const int32_t* scatter;  // rows of the output (of the gradient rows), or null
  void* out;
  int64_t ldo, stride_o;   // stride_o: of one expert's gradient
  int32_t E, rows, x_rows, out_rows;
  int32_t K, N, top;       // K: columns of x
  int32_t f_tiles, k_tiles;  // tiles of features; of x's features (gradient)
  int32_t kind;            // 0 fp16, 1 bf16
  int32_t out_dtype, pairs;  // pairs: two features of 16 bits at once
  uint32_t* status;
  uint64_t wait_limit_ns;
  int32_t inject_stall;
};

// Four rows r of 64 columns from x on, into 512 bytes of this CTA's shared memory.
__device__ __forceinline__ void tma_gather4_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int32_t x,
                                                 const int32_t (&r)[4]) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(r[0]), "r"(r[1]),
      "r"(r[2]), "r"(r[3])
      : "memory");
}

// A unit of work: one tile.
struct Unit {
  int expert, f0;      // expert, first feature of the pair's tile
  int first, count;    // its rows: sorted positions, or features of x (gradient)
  int width;           // count, rounded up to what an MMA takes
  int sum0, sum;       // gradient: the expert's sorted positions, summed over
};

// parts[e]: first unit of expert e; lo[e], n[e]: its sorted positions.
struct Table {
  const uint32_t* parts;
  const int32_t* lo;
  const int32_t* n;
};

__device__ __forceinline__ int row_tiles(int n) { return (n + MAX_ROWS - 1) / MAX_ROWS; }

template <int MODE>
__device__ __forceinline__ Unit unit_at(uint32_t u, const Params& p, const Table& t) {
  Unit w;
  if constexpr (MODE == GRADIENT) {
    const uint32_t per = p.f_tiles * p.k_tiles;
    const uint32_t e = u / per, r = u - e * per;
    w.expert = e;
    w.f0 = static_cast<int>(r % p.f_tiles) * TILE_F;
    w.first = static_cast<int>(r / p.f_tiles) * MAX_ROWS;
    w.count = min(MAX_ROWS, p.K - w.first);
    w.sum0 = t.lo[e];
    w.sum = t.n[e];
  } else {
    int e = 0, end = p.E;  // the last expert whose first unit is at most u
    while (end - e > 1) {
      const int mid = (e + end) >> 1;
      if (t.parts[mid] <= u)
        e = mid;
      else
        end = mid;
    }
    // an expert's rows in tiles of one size; its tiles of one weight tile follow one another
    const uint32_t r = u - t.parts[e], tiles = row_tiles(t.n[e]);
    const int size = ((t.n[e] + static_cast<int>(tiles) - 1) / static_cast<int>(tiles) + 31) & ~31;
    const int at = static_cast<int>(r % tiles) * size;
    w.expert = e;
    w.f0 = static_cast<int>(r / tiles) * TILE_F;
    w.first = t.lo[e] + at;
    w.count = max(0, min(size, t.n[e] - at));
    w.sum0 = 0;
    w.sum = p.K;
  }
  w.width = max(32, (w.count + 31) & ~31);
  return w;
}

// The output's rows of a warp's 32 columns of TMEM from row `first` on: lane j's row
// j, below 0 for none.
template <int MODE>
__device__ __forceinline__ int out_row(const Params& p, const Unit& w, int at, int lane) {
  if (at + lane >= w.count) return -1;
  const int r = w.first + at + lane;
  if (MODE == GRADIENT || !p.scatter) return r;
  const int s = p.scatter[r];
  return s < p.out_rows ? s : -1;
}

__device__ __forceinline__ uint32_t pack16(int dtype, uint32_t lo, uint32_t hi) {
  const float a = __uint_as_float(lo), b = __uint_as_float(hi);
  if (dtype == MHR_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 32 rows (columns of TMEM) of 32 features (lanes) to the output.
template <int MODE>
__device__ __forceinline__ void store_chunk(const uint32_t (&r)[32], const Params& p,
                                            const Unit& w, int at, int feature, int lane) {
  const int mine = out_row<MODE>(p, w, at, lane);
  const int rows = min(32, w.count - at);
  char* base = static_cast<char*>(p.out);
  if constexpr (MODE == GRADIENT)
    base += w.expert * p.stride_o * (p.out_dtype == MHR_F32 ? 4 : 2);
  if (p.out_dtype == MHR_F32) {
    float* out = reinterpret_cast<float*>(base) + feature;
    const bool in = feature < p.N;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int row = __shfl_sync(ALL, mine, j);
      if (j < rows && row >= 0 && in) out[row * p.ldo] = __uint_as_float(r[j]);
    }
  } else if (p.pairs) {
    // Neighbouring lanes exchange: the even one gets two features of row j, the odd
    // one of row j + 1, so that a store of the warp is two whole runs of 64 bytes.
    const int odd = lane & 1, f = feature - odd;
    uint16_t* out = reinterpret_cast<uint16_t*>(base) + f;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const uint32_t other = __shfl_xor_sync(ALL, odd ? r[j] : r[j + 1], 1);
      const uint32_t v = odd ? pack16(p.out_dtype, other, r[j + 1])
                             : pack16(p.out_dtype, r[j], other);
      const int row = __shfl_sync(ALL, mine, j + odd);
      if (j + odd < rows && row >= 0) {
        uint16_t* dst = out + row * p.ldo;
        if (f + 1 < p.N)
          *reinterpret_cast<uint32_t*>(dst) = v;
        else if (f < p.N)
          *dst = static_cast<uint16_t>(v);
      }
    }
  } else {
    uint16_t* out = reinterpret_cast<uint16_t*>(base) + feature;
    const bool in = feature < p.N;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int row = __shfl_sync(ALL, mine, j);
      if (j < rows && row >= 0 && in)
        out[row * p.ldo] = static_cast<uint16_t>(pack16(p.out_dtype, r[j], r[j]));
    }
  }
}

// Warp roles, barriers and the way a timeout unwinds are those of the other pair
// kernels (mxfp4_pair.cu): warp 0 producer, warp 1 MMA issuer (rank 0), warps 2-5
// epilogue; full[s] and released[b] in rank 0, empty[s] and acc_full[b] in both CTAs.
// tmW: the features' side.  tmX: x in boxes of 8 rows, or one for a gather; tmXBig:
// in boxes of 128 rows (no gather).
template <int MODE, bool GATHER>
__global__ void __launch_bounds__(THREADS, 1)
    routed_pair_kernel(const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ CUtensorMap tmXBig, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ alignas(8) uint64_t bars[2 * STAGES + 6];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ volatile uint32_t peer_loaded;          // rank 0: stages that rank 1 loaded
  __shared__ volatile uint32_t stage_tx[STAGES];     // bytes of a CTA's last load of a stage
  __shared__ volatile uint32_t peer_tx[STAGES];      // rank 0: rank 1's
  __shared__ uint32_t parts[MAX_PARTS + 1];
  __shared__ int32_t lo[MAX_PARTS], num[MAX_PARTS];
  __shared__ uint32_t sums[THREADS / 32];
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
  const uint32_t cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
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
    if (p.K > 0) {
      tma_prefetch_desc(&tmW);
      tma_prefetch_desc(&tmX);
      if (!GATHER) tma_prefetch_desc(&tmXBig);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  grid_dependency_wait();
  // The experts' parts, and the first unit of each.
  uint32_t units = 0;
  for (int e0 = 0; e0 < p.E; e0 += THREADS) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    uint32_t c = 0;
    if (e < p.E) {
      // (offsets that are not ascending, or past the rows, reach nothing)
      const int a = min(max(p.offsets[e], 0), p.rows), b = min(max(p.offsets[e + 1], a), p.rows);
      lo[e] = a;
      num[e] = b - a;
      c = MODE == GRADIENT ? p.f_tiles * p.k_tiles : row_tiles(b - a) * p.f_tiles;
    }
    uint32_t scan = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(ALL, scan, d);
      if (lane >= d) scan += o;
    }
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    uint32_t lower = 0, all = 0;
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) lower += sums[i];
      all += sums[i];
    }
    if (e < p.E) parts[e] = units + lower + scan - c;
    units += all;
    __syncthreads();
  }
  const Table table{parts, lo, num};
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint64_t limit = p.wait_limit_ns;

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
    for (uint32_t u = cluster; ok && u < units; u += clusters) {
      const Unit w = unit_at<MODE>(u, p, table);
      const int kbs = (w.sum + BK - 1) / BK, half = w.width / 2;
      const uint32_t tx = MODE == GRADIENT ? 2 * A_BYTES : A_BYTES + half * 128;
      const int f = w.f0 + static_cast<int>(rank) * HALF;
      const int mine = static_cast<int>(rank) * half;  // this CTA's first row of the tile
      int32_t r[4], g[4];  // this lane's four rows of x, and of the gradient rows
      if constexpr (MODE != GRADIENT && GATHER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = mine + 4 * lane + i;
          const int row = at < w.count ? p.gather[w.first + at] : -1;
          r[i] = row >= 0 && row / p.top < p.x_rows ? row / p.top : p.x_rows;
        }
      }
      for (int kb = 0; kb < kbs; ++kb, ++it) {
        if constexpr (MODE == GRADIENT) {  // (before the wait: the loads take their time)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = kb * BK + 4 * (lane & 15) + i;
            const bool in = at < w.sum;
            const int pos = w.sum0 + at;
            const int row = in ? (p.gather ? p.gather[pos] : pos) : -1;
            const int of = p.gather ? row / p.top : row;
            r[i] = row >= 0 && of < p.x_rows ? of : p.x_rows;
            const int to = in ? (p.scatter ? p.scatter[pos] : pos) : -1;
            g[i] = to >= 0 && to < p.out_rows ? to : p.out_rows;
          }
        }
        if (!__all_sync(ALL, mbar_wait_bounded(empty_bar(s), ph, limit, &abort_flag))) {
          if (lane == 0) give_up(kErrTimeoutProducer);
          ok = false;
          break;
        }
        const uint32_t st = sbase + s * STAGE_BYTES, fb = fb0 + 8u * s;
        if (lane == 0) {
          stage_tx[s] = tx;
          if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * tx);
        }
        __syncwarp();
        if (!(stall && it == 0)) {
          if constexpr (MODE == GRADIENT) {
            // 64 positions x 64 features a box: lanes 0-15 the first box, 16-31 the second
            const int box = lane >> 4;
            const uint32_t to = st + box * BOX + (lane & 15) * 512;
            tma_gather4_pair(to, &tmW, fb, f + 64 * box, g);
            tma_gather4_pair(to + A_BYTES, &tmX, fb, w.first + mine + 64 * box, r);
          } else {
            if (elect_one()) {
              if constexpr (MODE == PRODUCT) {
                tma_load_3d_pair(st, &tmW, fb, f, kb * BK, w.expert);
                tma_load_3d_pair(st + BOX, &tmW, fb, f + 64, kb * BK, w.expert);
              } else {
                tma_load_3d_pair(st, &tmW, fb, kb * BK, f, w.expert);
              }
            }
            if constexpr (GATHER) {
              if (4 * lane < half)
                tma_gather4_pair(st + A_BYTES + lane * 512, &tmX, fb, kb * BK, r);
            } else if (half == HALF) {
              if (elect_one())
                tma_load_2d_pair(st + A_BYTES, &tmXBig, fb, kb * BK, w.first + mine);
            } else if (8 * lane < half) {
              tma_load_2d_pair(st + A_BYTES + lane * 1024, &tmX, fb, kb * BK,
                               w.first + mine + 8 * lane);
            }
          }
        }
        __syncwarp();
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (lane == 0) {
      // Both CTAs' loads complete in rank 0, which waits for all of them -- counting as
      // done what either side never issued -- before either CTA may leave.
      volatile int never = 0;
      if (!leader) {
        for (int i = 0; i < STAGES; ++i)
          st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t*>(peer_tx + i)), 0),
                                stage_tx[i]);
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
        for (uint32_t i = hi > STAGES ? hi - STAGES : 0; i < hi; ++i) {
          const uint32_t si = i % STAGES, phi = (i / STAGES) & 1u;
          const bool armed = i < it, loaded0 = armed && !(stall && i == 0), loaded1 = i < it1;
          if (!armed) {
            mbar_arrive_expect_tx(full_bar(si), peer_tx[si]);
          } else {
            const uint32_t missing =
                (loaded0 ? 0u : stage_tx[si]) + (loaded1 ? 0u : stage_tx[si]);
            if (missing) {  // once the MMA issuer has given up on the stage
              mbar_wait_bounded(full_bar(si), phi, 2 * limit, &abort_flag);
              mbar_complete_tx(full_bar(si), missing);
            }
          }
          if (!mbar_wait_bounded(full_bar(si), phi, limit, &never))
            atomicOr(p.status, kErrTimeoutDrain);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader) {
      uint32_t it = 0, t = 0, s = 0, ph = 0;
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {  // a warp-uniform outcome
        return __all_sync(ALL, mbar_wait_bounded(bar, parity, limit, &abort_flag)) != 0;
      };
      for (uint32_t u = cluster; ok && u < units; u += clusters, ++t) {
        const Unit w = unit_at<MODE>(u, p, table);
        const int kbs = (w.sum + BK - 1) / BK;
        const int tail = (w.sum - (kbs - 1) * BK + 15) / 16;  // MMAs of the last stage
        const uint32_t idesc =
            make_idesc(p.kind, MODE != TRANSPOSED, MODE == GRADIENT, TILE_F, w.width);
        if (t >= 2 && !wait(released_bar(t & 1u), ((t - 2) >> 1) & 1u)) {
          if (lane == 0) give_up(kErrTimeoutMma);
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (t & 1u) * MAX_ROWS;
        for (int kb = 0; kb < kbs; ++kb, ++it) {
          if (!wait(full_bar(s), ph)) {
            if (lane == 0) give_up(kErrTimeoutMma);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = sbase + s * STAGE_BYTES;
          const uint64_t a = MODE == TRANSPOSED ? smem_desc_sw128(st, 16, 1024)
                                                : smem_desc_sw128(st, BOX, 1024);
          const uint64_t b = MODE == GRADIENT ? smem_desc_sw128(st + A_BYTES, BOX, 1024)
                                              : smem_desc_sw128(st + A_BYTES, 16, 1024);
          // 16 of the sum: 32 bytes along a K-major row, 16 rows of 128 bytes else
          constexpr uint32_t step_a = (MODE == TRANSPOSED ? 32 : 2048) >> 4;
          constexpr uint32_t step_b = (MODE == GRADIENT ? 2048 : 32) >> 4;
          const int mmas = kb + 1 < kbs ? BK / 16 : tail;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              if (kk < mmas)
                mma_f16_pair(d, a + kk * step_a, b + kk * step_b, idesc, kb > 0 || kk > 0 ? 1u : 0u);
            mma_commit_pair_multicast(empty_bar(s), 0x3);
            if (kb + 1 == kbs) mma_commit_pair_multicast(acc_bar(t & 1u), 0x3);
          }
          __syncwarp();
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (kbs == 0 && elect_one()) mma_commit_pair_multicast(acc_bar(t & 1u), 0x3);
        __syncwarp();
      }
      if (elect_one()) mma_commit_pair(drain_bar);
      __syncwarp();
      volatile int never = 0;
      if (!mbar_wait_bounded(drain_bar, 0, limit, &never) && lane == 0)
        atomicOr(p.status, kErrTimeoutDrain);
    }
    __syncwarp();
  } else {
    const int q = warp & 3;
    uint32_t t = 0;
    for (uint32_t u = cluster; u < units; u += clusters, ++t) {
      const uint32_t b = t & 1u;
      const Unit w = unit_at<MODE>(u, p, table);
      if (!__all_sync(ALL, mbar_wait_bounded(acc_bar(b), (t >> 1) & 1u, limit, &abort_flag, 128))) {
        if (lane == 0) give_up(kErrTimeoutEpilogue);
        __syncwarp();
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + b * MAX_ROWS;
      const int feature = w.f0 + static_cast<int>(rank) * HALF + q * 32 + lane;
#pragma unroll 1
      for (int at = 0; at < w.count; at += 32) {
        uint32_t r[32];
        tmem_ld_32cols(taddr + at, r);
        tmem_ld_wait();
        if (w.sum == 0) {  // no terms: the accumulator was not written
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0;
        }
        if (at + 32 >= w.count) {  // all read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(released_bar(b), 0));
        }
        store_chunk<MODE>(r, p, w, at, feature, lane);
      }
      if (w.count <= 0 && lane == 0) mbar_arrive_cluster(mapa_shared(released_bar(b), 0));
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

// An operand whose rows TMA cannot read, row by row into scratch with a pitch of
// whole 16 bytes; parts (experts) without rows of tokens are left out where
// `offsets` is given.
__global__ void repack_kernel(const uint16_t* src, int64_t rows, int64_t cols, int64_t ld,
                              int64_t stride, const int32_t* offsets, uint16_t* dst,
                              int64_t dst_ld) {
  const int64_t part = blockIdx.y;
  if (offsets && offsets[part + 1] <= offsets[part]) return;
  src += part * stride;
  dst += part * rows * dst_ld;
  const int lanes = 32, warp = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x / lanes);
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (blockDim.x / lanes) + warp; r < rows;
       r += warps)
    for (int64_t c = lane; c < cols; c += lanes) dst[r * dst_ld + c] = src[r * ld + c];
}

struct Ready {
  const void* p;
  int64_t ld, stride;
};

// The operand as TMA reads it: itself, or a copy at *scratch, which moves on.
cudaError_t ready(const void* p, int64_t parts, int64_t rows, int64_t cols, int64_t ld,
                  int64_t stride, const int32_t* offsets, char** scratch, cudaStream_t s,
                  Ready* out) {
  if (repack_bytes(p, parts, rows, cols, ld, stride) == 0) {
    *out = {p, ld, stride};
    return cudaSuccess;
  }
  const int64_t dst_ld = (cols + 7) / 8 * 8;
  uint16_t* dst = reinterpret_cast<uint16_t*>(*scratch);
  *out = {dst, dst_ld, rows * dst_ld};
  *scratch += repack_bytes(p, parts, rows, cols, ld, stride);
  const int64_t blocks = (rows + 7) / 8;
  const dim3 grid(static_cast<unsigned>(blocks < 1024 ? blocks : 1024),
                  static_cast<unsigned>(parts));
  repack_kernel<<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(p), rows, cols, ld, stride,
                                     offsets, dst, dst_ld);
  note_launch();
  return cudaGetLastError();
}

template <int MODE, bool GATHER>
cudaError_t launch_t(const CUtensorMap (&m)[3], const Params& p, cudaLaunchConfig_t cfg) {
  auto kern = routed_pair_kernel<MODE, GATHER>;
  static int most[64];  // by device; under the library's lock
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  int clusters = device < 64 ? most[device] : 0;
  if (!clusters) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM)) !=
        cudaSuccess)
      return e;
    cfg.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg)) != cudaSuccess) return e;
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    if (device < 64) most[device] = clusters;
  }
  // As many units as there can be at most: every row tile but one of an expert's full.
  const int64_t tiles = MODE == GRADIENT
                            ? static_cast<int64_t>(p.E) * p.k_tiles
                            : (p.rows < p.E ? p.rows : p.E) + p.rows / MAX_ROWS;
  const int64_t units = tiles * p.f_tiles;
  if (units > 0x3fffffff) return cudaErrorInvalidConfiguration;
  if (units < clusters) clusters = static_cast<int>(units);
  cfg.gridDim = dim3(2 * clusters);
  cfg.numAttrs = 2;
  note_main_kernel(MODE == GRADIENT     ? "routed_pair_kernel<gradient>"
                   : MODE == TRANSPOSED ? "routed_pair_kernel<transposed>"
                                        : "routed_pair_kernel<product>",
                   2 * clusters, static_cast<int>(units));
  e = cudaLaunchKernelEx(&cfg, kern, m[0], m[1], m[2], p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int64_t repack_bytes(const void* p, int64_t parts, int64_t rows, int64_t cols, int64_t ld,
                     int64_t stride) {
  if (rows == 0 || cols == 0 ||
      (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows == 1 || ld % 8 == 0) &&
       (parts == 1 || stride % 8 == 0)))
    return 0;
  int64_t n;
  if (__builtin_mul_overflow(parts * rows, (cols + 7) / 8 * 16, &n) || n > INT64_MAX - 255)
    return -1;
  return (n + 255) / 256 * 256;
}

cudaError_t launch_product(const ProductArgs& a, void* scratch, const DeviceCtl& ctl,
                           cudaStream_t s) {
  const bool gradient = a.kind == ProductKind::gradient;
  Params p;
  p.offsets = a.offsets;
  p.gather = a.gather;
  p.scatter = a.scatter;
  p.out = a.out;
  p.ldo = a.ldo;
  p.stride_o = a.stride_o;
  p.E = static_cast<int32_t>(a.E);
  p.rows = static_cast<int32_t>(a.rows);
  p.x_rows = static_cast<int32_t>(a.x_rows);
  p.out_rows = static_cast<int32_t>(a.out_rows);
  // (a sum over nothing, or over rows that are not there, is zero)
  const bool none = gradient ? a.rows == 0 || a.x_rows == 0 || a.out_rows == 0
                             : a.K == 0 || a.x_rows == 0;
  p.K = static_cast<int32_t>(none && !gradient ? 0 : a.K);
  if (none && gradient) p.rows = 0;
  p.N = static_cast<int32_t>(a.N);
  p.top = static_cast<int32_t>(a.top);
  p.f_tiles = static_cast<int32_t>((a.N + TILE_F - 1) / TILE_F);
  p.k_tiles = static_cast<int32_t>((a.K + MAX_ROWS - 1) / MAX_ROWS);
  p.kind = a.dtype == MHR_BF16 ? 1 : 0;
  p.out_dtype = a.out_dtype;
  p.pairs = a.out_dtype != MHR_F32 && reinterpret_cast<uintptr_t>(a.out) % 4 == 0 &&
            a.ldo % 2 == 0 && (!gradient || a.stride_o % 2 == 0);
  p.status = ctl.status;
  p.wait_limit_ns = ctl.wait_limit_ns;
  p.inject_stall = ctl.inject_stall;

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

  CUtensorMap m[3] = {};
  const auto type = a.dtype == MHR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const auto swizzle = CU_TENSOR_MAP_SWIZZLE_128B;
  if (!none) {
    char* at = static_cast<char*>(scratch);
    Ready x, w;
    cudaError_t e = ready(a.x, 1, a.x_rows, a.K, a.ldx, 0, nullptr, &at, s, &x);
    if (e != cudaSuccess) return e;
    auto rows_map = [&](CUtensorMap* map, const Ready& r, int64_t cols, int64_t rows,
                        uint32_t box) {
      // (one row has no pitch of its own to go by)
      const int64_t ld = rows == 1 ? (cols + 7) / 8 * 8 : r.ld;
      return encode_tmap_2d(map, type, r.p, cols, rows, ld * 2, 64, box, swizzle) == CUDA_SUCCESS;
    };
    bool ok = true;
    if (gradient) {
      e = ready(a.w, 1, a.out_rows, a.N, a.ldw, 0, nullptr, &at, s, &w);
      if (e != cudaSuccess) return e;
      ok = rows_map(&m[0], w, a.N, a.out_rows, 1) && rows_map(&m[1], x, a.K, a.x_rows, 1);
    } else {
      const bool t = a.kind == ProductKind::transposed;
      const int64_t rows = t ? a.N : a.K, cols = t ? a.K : a.N;
      e = ready(a.w, a.E, rows, cols, a.ldw, a.stride_w, a.offsets, &at, s, &w);
      if (e != cudaSuccess) return e;
      const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows),
                                static_cast<uint64_t>(a.E)};
      const int64_t ld = rows == 1 ? (cols + 7) / 8 * 8 : w.ld;
      const int64_t stride = a.E == 1 ? rows * ((cols + 7) / 8 * 8) : w.stride;
      const uint64_t pitch[2] = {static_cast<uint64_t>(ld) * 2, static_cast<uint64_t>(stride) * 2};
      const uint32_t box[3] = {64, t ? 128u : 64u, 1};
      ok = encode_tmap_3d(&m[0], type, w.p, dims, pitch, box, swizzle) == CUDA_SUCCESS &&
           rows_map(&m[1], x, a.K, a.x_rows, a.gather ? 1 : 8) &&
           (a.gather || rows_map(&m[2], x, a.K, a.x_rows, 128));
    }
    if (!ok) return cudaErrorInvalidValue;
  }
  MainKernelEvents ev(s);
  switch (a.kind) {
    case ProductKind::gradient: return launch_t<GRADIENT, true>(m, p, cfg);
    case ProductKind::transposed:
      return a.gather ? launch_t<TRANSPOSED, true>(m, p, cfg)
                      : launch_t<TRANSPOSED, false>(m, p, cfg);
    default:
      return a.gather ? launch_t<PRODUCT, true>(m, p, cfg) : launch_t<PRODUCT, false>(m, p, cfg);
  }
}

}  // namespace routed
}  // namespace mhr
