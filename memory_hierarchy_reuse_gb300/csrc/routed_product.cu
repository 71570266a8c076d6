// The experts' products (gemm_routed_product) and their weights' gradient
// (gemm_routed_weight_grad): persistent CTA pairs (tcgen05 cta_group::2).
//
// A product's tile has the output's columns -- features -- on the MMA's rows, 256 of
// them, and rows of tokens on its columns, 32 to 256: an expert's rows are few and of
// any number, its features many, so the side that varies is the one whose length an MMA
// takes in steps.  The transposed result costs nothing: a lane of TMEM is a feature, so a
// warp's store of one row is 32 neighbours.  A gradient's tile has x's features on the
// MMA's rows and the gradient's, up to 256 of them, on its columns: a lane holds a row of
// the result, and its neighbours go out as rows of 128 bytes.  Which tiles there are stands in the offsets on the device alone; every
// CTA sums them up in shared memory and takes every clusters-th.
//
// Operands:          features side               rows side
//   product           W_e (K x N): MN-major       x rows, K-major
//   transposed        W_e (N x K): K-major        x rows, K-major
//   weight gradient   x rows, MN-major            gradient rows, MN-major
// All come by TMA.  Rows that an index picks are put in order first by a kernel of their
// own; of few rows, TMA's gather of four rows brings them, a lane four rows.  (The gather
// takes some 60 cycles for its 512 bytes: 8192 tokens, 8 of 16 experts of 4096 x 4096,
// 4283 us with it against 1143 for rows in order; copies by the threads into the same
// layout were as slow.)  A row outside its matrix -- past an expert's last, or an index
// out of range -- is zeros.
//
// GB300: few rows are bound by the weights' bytes (30 tokens, 8 of 128 experts of 2048 x
// 1536: 100 us, 6.7 TB/s; one token 12.2 us), and so are up to 128 rows an expert (4096 x
// 1536: 262 us, 6.9 TB/s, 790 TFLOP/s); at 256 rows 1.2 to 1.4 PFLOP/s.  The gradient of 64
// experts of 2048 x 1408 in fp32: 179 us of sorted rows, of which the stores alone are 123.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdio>
#include <type_traits>

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
// Of the sum a stage: two swizzle rows of 128 bytes.  A stage costs the issuing warps some
// 300 cycles whatever it holds; with 64 an MMA of few rows was done long before (319 MB of
// weights for eight rows in 105 us).
constexpr int BK = 128;
constexpr int A_BYTES = HALF * BK * 2;       // this CTA's features
constexpr int BOX = 128 * 128;               // 128 rows of 128 bytes
constexpr int MAX_STAGES = 6;
constexpr int EPI_WARPS = 8;
constexpr int CLASSES = 8;                   // of experts, by what their units cost
constexpr int THREADS = 32 * (3 + EPI_WARPS);

enum Mode { PRODUCT = 0, TRANSPOSED = 1, GRADIENT = 2 };

// LONG: fp32 results.  The tensor cores add into their fp32 accumulators by truncation,
// which takes 1.4e-8 of a sum off with its first 16 terms, 3e-7 after 256 and 1.7e-6 after
// 1024 (means of sums of positive terms, GB300): the sum goes on in registers, rounded
// to nearest, after every SEGMENT stages.  16-bit results, up to 4e-3 or 5e-4 off by their
// own rounding, do without.  An epilogue thread holds 64 of a tile's 128 columns.
template <bool LONG>
struct Shape {
  static constexpr int ROWS = LONG ? 128 : 256;            // rows of a pair's tile, at most
  static constexpr int B_BYTES = ROWS / 2 * BK * 2;        // this CTA's half of them
  static constexpr int RING_BYTES = LONG ? 168 * 1024 : 192 * 1024;
  static constexpr int SEGMENT = LONG ? 3 : 1 << 30;       // stages an accumulator takes
  static constexpr int PIECE_BYTES = 32 * 32 * (LONG ? 4 : 2);  // of an epilogue warp (of two,
                                                                // of a 16-bit gradient)
  static constexpr int SMEM = RING_BYTES + EPI_WARPS * PIECE_BYTES + 1024;
  static constexpr uint32_t TMEM_COLS = 2 * ROWS;
};

struct Params {
  const int32_t* offsets;
  const int32_t* gather;   // rows of x over `top`, or null
  const int32_t* scatter;  // rows of the output, or null
  void* out;
  int64_t ldo, stride_o;   // stride_o: of one expert's gradient
  int32_t E, rows, x_rows, out_rows;
  int32_t K, N, top;       // K: columns of x
  int32_t f_tiles, n_tiles;  // tiles of features; of the gradient's features on the other side
  int32_t kind;            // 0 fp16, 1 bf16
  int32_t out_dtype;
  int32_t out_tma, pairs;  // whole chunks by TMA; else two features of 16 bits at once
  uint32_t* status;
  uint64_t wait_limit_ns;
  int32_t inject_stall;
};

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t x,
                                             int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(x), "r"(y), "r"(z)
      : "memory");
}

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

// The features' side in boxes of 16 to 128 rows (gradient), or whatever a product's
// weights take (w[3]); x in boxes of 16 to 128 rows; either in single rows for a gather.
// A TMA instruction takes some 60 cycles however little it brings, so rows come in a few
// boxes of powers of two (4096 tokens, 8 of 128 experts of 1536 x 4096 with skewed
// counts: 562 us with boxes of 8 rows).
struct Maps {
  CUtensorMap w[4], x[4], w1, x1, out;  // out: in boxes of an epilogue warp's chunk
};

// A value that all lanes of a warp have, for a uniform register: what a TMA or an MMA takes
// from others costs its warp some hundred cycles an instruction to bring there.
__device__ __forceinline__ int same(int v) { return __shfl_sync(ALL, v, 0); }

// mma_f16_pair by the low words of the descriptors: the address and the leading offset.
__device__ __forceinline__ uint32_t desc_word(uint32_t saddr, uint32_t lbo_bytes) {
  return ((saddr & 0x3FFFFu) >> 4) | (lbo_bytes >> 4) << 16;
}
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(mx::DESC_HI_SW128)
      : "memory");
}

// A unit of work: one tile.
struct Unit {
  int expert, f0;      // expert, first feature of the pair's tile
  int first, count;    // its rows: sorted positions, or columns of the output (gradient)
  int width;           // count, rounded up to what an MMA takes
  int sum0, sum;       // gradient: the expert's sorted positions, summed over
};

// Experts in descending order of what their units cost: expert[i] has the units from
// parts[i] on (parts has one more); its sorted positions are n[e] from lo[e] on.
struct Table {
  const uint32_t* parts;
  const int32_t* expert;
  const int32_t* lo;
  const int32_t* n;
};

// n / d; of n that a float holds, by its quotient, which is off by one at most.
__device__ __forceinline__ uint32_t divide(uint32_t n, uint32_t d) {
  if (n >= 1u << 22 || d == 0) return d ? n / d : 0;
  uint32_t q = __float2uint_rz(__fdividef(static_cast<float>(n), static_cast<float>(d)));
  if (q * d > n) --q;
  if (n - q * d >= d) ++q;
  return q;
}

template <int ROWS>
__device__ __forceinline__ int row_tiles(int n) {
  return (n + ROWS - 1) / ROWS;
}
// Rows of an expert's tiles: all of one size.
template <int ROWS>
__device__ __forceinline__ int tile_rows(int n) {
  const int tiles = row_tiles<ROWS>(n);
  if (tiles <= 1) return max(32, (n + 31) & ~31);
  return (static_cast<int>(divide(n + tiles - 1, tiles)) + 31) & ~31;
}

// How much a unit of an expert of n rows costs: the steps of an MMA's columns; of a
// gradient, the stages, by powers of two.  Clusters take units in turn, the dearest
// first, so that two clusters' work differs by one unit's at most (in turn in the
// experts' order, clusters of skewed counts were up to a fifth apart).  Runs of units
// of like cost for each cluster would be as even, but scatter the experts over time:
// 8192 tokens, 8 of 16 experts of 4096 x 4096, 2624 us against 1143, from HBM.
template <int MODE, int ROWS>
__device__ __forceinline__ int cost_class(int n) {
  if (n == 0) return 0;
  if constexpr (MODE == GRADIENT) return min(CLASSES - 1, 32 - __clz((n + BK - 1) / BK));
  return tile_rows<ROWS>(n) * CLASSES / ROWS - 1;
}

// Unit u, found by a whole warp from its place in the table on (a warp's units ascend:
// looked up among all experts, each took 550 cycles).
template <int MODE, int ROWS>
__device__ __forceinline__ Unit unit_at(uint32_t u, const Params& p, const Table& t, int& place) {
  const int lane = threadIdx.x & 31;
  int i = place;
  for (int behind = 32; behind == 32; i += behind) {  // the last place with a first unit <= u
    const int at = i + 1 + lane;
    behind = __popc(__ballot_sync(ALL, at < p.E && t.parts[at] <= u));
  }
  place = i;
  const int e = t.expert[i];
  Unit w;
  const uint32_t r = u - t.parts[i];
  w.expert = e;
  if constexpr (MODE == GRADIENT) {
    const uint32_t q = divide(r, p.f_tiles);
    w.f0 = static_cast<int>(r - q * p.f_tiles) * TILE_F;
    w.first = static_cast<int>(q) * ROWS;
    w.count = min(ROWS, p.N - w.first);
    w.sum0 = t.lo[e];
    w.sum = t.n[e];
  } else {
    const int tiles = row_tiles<ROWS>(t.n[e]), size = tile_rows<ROWS>(t.n[e]);
    const uint32_t q = divide(r, tiles);
    const int at = static_cast<int>(r - q * tiles) * size;
    w.f0 = static_cast<int>(q) * TILE_F;
    w.first = t.lo[e] + at;
    w.count = max(0, min(size, t.n[e] - at));
    w.sum0 = 0;
    w.sum = p.K;
  }
  w.width = max(32, (w.count + 31) & ~31);
  return w;
}

// The row that an index picks, over `top`: below 0 where it lies outside `rows`.
__device__ __forceinline__ int picked_row(int index, int top, int rows) {
  const int r = index >= 0 ? index / top : -1;
  return r < rows ? r : -1;
}

template <int DTYPE>
__device__ __forceinline__ uint32_t pack16(uint32_t lo, uint32_t hi) {
  const float a = __uint_as_float(lo), b = __uint_as_float(hi);
  if constexpr (DTYPE == MHR_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 32 rows (columns of TMEM) of 32 features (lanes) to the output: of fp32 (WIDE), or of
// 16 bits.  Whole chunks by TMA from the warp's piece of shared memory: a store of a lane's
// own values, or of 16 bytes a lane, holds the SM up 5 to 10 cycles for every 128 bytes.
// No branch a row either way -- for the row, for the type, for the lane's parity -- which
// cost 2700 cycles a chunk.
template <bool WIDE>
__device__ __forceinline__ void store_chunk(const uint32_t (&r)[32], const Params& p,
                                            const CUtensorMap* out_map, uint32_t piece,
                                            const Unit& w, int at, int feature, int lane) {
  using Word = std::conditional_t<WIDE, uint32_t, uint16_t>;
  Word* base = static_cast<Word*>(p.out);
  const int count = min(32, w.count - at);  // rows of this chunk
  const bool scattered = p.scatter != nullptr;
  const int first = w.first + at;
  int mine = first + lane;  // lane j's row of the output, below 0 for none
  if (scattered) mine = lane < count ? picked_row(p.scatter[first + lane], 1, p.out_rows) : -1;
  // Pairs: neighbouring lanes exchange, the even one gets two features of row j, the odd
  // one of row j + 1, so that a store of the warp is two runs of 64 bytes.
  const bool pairs = !WIDE && p.pairs;  // (as where chunks go by TMA)
  const int odd = pairs ? lane & 1 : 0, each = pairs ? 2 : 1, f = feature - odd;
  uint32_t v[WIDE ? 1 : 16];
  if constexpr (!WIDE) {
    if (pairs) {
#pragma unroll
      for (int j = 0; j < 32; j += 2) v[j / 2] = __shfl_xor_sync(ALL, odd ? r[j] : r[j + 1], 1);
      auto pack = [&](auto dtype) {
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const uint32_t lo = odd ? v[j / 2] : r[j], hi = odd ? r[j + 1] : v[j / 2];
          v[j / 2] = pack16<decltype(dtype)::value>(lo, hi);
        }
      };
      if (p.out_dtype == MHR_BF16)
        pack(std::integral_constant<int, MHR_BF16>{});
      else
        pack(std::integral_constant<int, MHR_F16>{});
    }
  }
  // (the rows behind a tile's are another's)
  if (p.out_tma && !scattered && count == 32) {
    if (lane == 0) bulk_wait_group_read<0>();  // the chunk before has left the piece
    __syncwarp();
    if constexpr (WIDE) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(piece + j * 128 + lane * 4), "r"(r[j])
                     : "memory");
    } else {
#pragma unroll
      for (int j = 0; j < 32; j += 2)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(piece + (j + odd) * 64 + (lane - odd) * 2),
                     "r"(v[j / 2])
                     : "memory");
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && f < p.N) {
      tma_store_3d(out_map, piece, f, first, 0);
      bulk_commit_group();
    }
    return;
  }
  if (WIDE || pairs) {
    const bool in = f + each <= p.N;
#pragma unroll
    for (int j0 = 0; j0 < 32; j0 += WIDE ? 8 : 16) {
      int to[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = j0 + i * (WIDE ? 1 : 2);
        to[i] = __shfl_sync(ALL, mine, j + odd);
        if (j + odd >= count || !in) to[i] = -1;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        Word* dst = base + to[i] * p.ldo + f;
        if (to[i] >= 0) {
          if constexpr (WIDE)
            *dst = r[j0 + i];
          else
            *reinterpret_cast<uint32_t*>(dst) = v[j0 / 2 + i];
        }
      }
    }
    if constexpr (!WIDE) {
      if (__any_sync(ALL, f + 1 == p.N)) {  // the last of an odd number of features
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int to = __shfl_sync(ALL, mine, 2 * i + odd);
          if (f + 1 == p.N && 2 * i + odd < count && to >= 0)
            base[to * p.ldo + f] = static_cast<uint16_t>(v[i]);
        }
      }
    }
  } else {
    const bool in = feature < p.N;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int to = __shfl_sync(ALL, mine, j);
      if (j < count && to >= 0 && in) {
        const float x = __uint_as_float(r[j]);
        base[to * p.ldo + feature] = static_cast<Word>(
            p.out_dtype == MHR_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x))
                                    : __half_as_ushort(__float2half_rn(x)));
      }
    }
  }
}

// A gradient's chunk of 32 rows and 32 columns where TMA cannot write it, from the warp's
// piece on: rows 4 bytes a lane, no branch a row.  Of 16 bits a row may start between two
// words: then a lane's word is its second value and its neighbour's first, and the row's
// ends go out as 2 bytes.  (Inlined, it slowed results that TMA writes: the gradient of 64
// experts of 2048 x 1408 in fp32 197 -> 235 us.)
__device__ __noinline__ void store_ragged(uint32_t* to, int64_t ldo, int rows, int cols,
                                          uint32_t piece, int lane) {
  const int last = lane < cols ? rows : 0;
#pragma unroll
  for (int j0 = 0; j0 < 32; j0 += 8) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      asm volatile("ld.shared.b32 %0, [%1];"
                   : "=r"(w[i])
                   : "r"(piece + (j0 + i) * 128 + (((lane >> 2) ^ i) << 4) + (lane & 3) * 4)
                   : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i, to += ldo)
      if (j0 + i < last) to[lane] = w[i];
  }
}
__device__ __noinline__ void store_ragged(uint16_t* to, int64_t ldo, int rows, int cols,
                                          uint32_t piece, int lane) {
  const int sub = lane >> 4, l = lane & 15;  // two rows at once
  to += sub * ldo;
#pragma unroll
  for (int j0 = 0; j0 < 32; j0 += 16) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      asm volatile("ld.shared.b32 %0, [%1];"
                   : "=r"(w[i])
                   : "r"(piece + (j0 + 2 * i + sub) * 64 + (((l >> 2) ^ (i & 3)) << 4) + (l & 3) * 4)
                   : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i, to += 2 * ldo) {
      const uint32_t next = __shfl_down_sync(ALL, w[i], 1, 16);
      const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(to) >> 1 & 1);
      const int first = 2 * l + shift;  // of the word's two columns
      const bool in = j0 + 2 * i + sub < rows;
      if (in && first + 1 < cols)
        *reinterpret_cast<uint32_t*>(to + first) = __funnelshift_r(w[i], next, 16 * shift);
      // what is left over: the first column, and the last one
      const bool head = in && shift && l == 0, tail = in && first + 1 == cols;
      if (head || tail)
        to[head ? 0 : first] = static_cast<uint16_t>(head ? w[i] : w[i] >> (16 * shift));
      if (head && tail) to[first] = static_cast<uint16_t>(w[i] >> 16);
    }
  }
}

// A gradient's 32 rows (lanes, from `row` on) of 128 bytes of columns from `col` on, by way
// of the warp's piece of shared memory, swizzled.
__device__ __forceinline__ void store_rows(const uint32_t (&v)[32], const Params& p,
                                           const CUtensorMap* out_map, uint32_t piece, int expert,
                                           int row, int col, int lane) {
  if (p.out_tma) {  // (the store before has left the piece)
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(piece + lane * 128 +
                                                                 ((k ^ (lane & 7)) << 4)),
                 "r"(v[4 * k]), "r"(v[4 * k + 1]), "r"(v[4 * k + 2]), "r"(v[4 * k + 3])
                 : "memory");
  if (p.out_tma) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && row < p.K && col < p.N) {
      tma_store_3d(out_map, piece, col, row, expert);
      bulk_commit_group();
    }
    return;
  }
  __syncwarp();  // (fp32: a 16-bit gradient's ragged rows go another way)
  store_ragged(static_cast<uint32_t*>(p.out) + expert * p.stride_o + row * p.ldo + col, p.ldo,
               min(32, p.K - row), min(32, p.N - col), piece, lane);
  __syncwarp();
}

// Warp roles, barriers and the way a timeout unwinds are those of the other pair
// kernels (mxfp4_pair.cu): warps 0 and 10 producers, of either side, warp 1 MMA issuer
// (rank 0), warps 2-9 epilogue; full[.][s] and released[b] in rank 0, empty[s] and acc_full[b] in both CTAs.
// Rank 1's epilogue hands an accumulator back to its own read[b], from where its warp 1,
// idle otherwise, tells rank 0: an arrival that is released to the cluster waits for the
// stores that its thread has under way.
template <int MODE, bool INDEXED, bool LONG>
__global__ void __launch_bounds__(THREADS, 1)
    routed_pair_kernel(const __grid_constant__ Maps maps, const Params p) {
  using S = Shape<LONG>;
  constexpr int ROWS = S::ROWS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ alignas(8) uint64_t bars[3 * MAX_STAGES + 9];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  // Of either side (0: features, 1: rows):
  __shared__ volatile uint32_t peer_loaded[2];        // rank 0: stages that rank 1 loaded
  __shared__ volatile uint32_t stage_tx[2][MAX_STAGES];   // bytes of a CTA's last load of a stage
  __shared__ volatile uint32_t other_tx[2][MAX_STAGES];   // rank 0: and of rank 1's with it
  __shared__ volatile uint32_t peer_tx[2][MAX_STAGES];    // rank 0: rank 1's
  __shared__ uint32_t parts[MAX_PARTS + 1];
  __shared__ int32_t expert[MAX_PARTS], lo[MAX_PARTS], num[MAX_PARTS];
  __shared__ uint32_t class_units[CLASSES], class_experts[CLASSES];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem), bar0 = smem_u32(bars);
  auto full_bar = [&](int side, uint32_t s) { return bar0 + 8u * (side * MAX_STAGES + s); };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (2 * MAX_STAGES + s); };
  auto acc_bar = [&](uint32_t b) { return bar0 + 8u * (3 * MAX_STAGES + b); };
  auto released_bar = [&](uint32_t b) { return bar0 + 8u * (3 * MAX_STAGES + 2 + b); };
  auto read_bar = [&](uint32_t b) { return bar0 + 8u * (3 * MAX_STAGES + 4 + b); };
  const uint32_t drain_bar = bar0 + 8u * (3 * MAX_STAGES + 6);
  auto peer_done_bar = [&](int side) { return bar0 + 8u * (3 * MAX_STAGES + 7 + side); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  const uint32_t peer_abort = mapa_shared(smem_u32(const_cast<int*>(&abort_flag)), rank ^ 1u);

  if (threadIdx.x == 0) {
    for (int s = 0; s < MAX_STAGES; ++s) {
      mbar_init(full_bar(0, s), 1);
      mbar_init(full_bar(1, s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_bar(b), 1);
      mbar_init(released_bar(b), EPI_WARPS + 1);
      mbar_init(read_bar(b), EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    for (int side = 0; side < 2; ++side) {
      mbar_init(peer_done_bar(side), 1);
      peer_loaded[side] = 0;
    }
    abort_flag = 0;
    fence_mbar_init();
    if (p.K > 0 && p.rows > 0) {  // (else there are no maps)
      tma_prefetch_desc(&maps.w[3]);
      for (int i = 0; i < 4; ++i) tma_prefetch_desc(&maps.x[i]);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&tmem_slot), S::TMEM_COLS);
    tmem_relinquish_pair();
  }
  if (threadIdx.x < CLASSES) class_units[threadIdx.x] = class_experts[threadIdx.x] = 0;
  __syncthreads();
  grid_dependency_wait();
  // The experts' rows, then their places: a warp takes a class, whose place is behind
  // the dearer ones.
  auto units_of = [&](int n) -> uint32_t {
    return (MODE == GRADIENT ? p.n_tiles : row_tiles<ROWS>(n)) * p.f_tiles;
  };
  auto scan_of = [&](uint32_t c) {
    uint32_t scan = c;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const uint32_t o = __shfl_up_sync(ALL, scan, i);
      if (lane >= i) scan += o;
    }
    return scan;
  };
  bool few = MODE != GRADIENT && p.rows <= FEW_ROWS;
  bool falls = false;  // an offset that this thread has seen lies below the one before
  if (few) {
    // Units of like cost: in the experts' order, by one warp, 128 offsets at a time.
    if (warp == 0) {
      uint32_t unit = 0;
      int dearest = 0;
      for (int e0 = 0; e0 < p.E; e0 += 128) {
        int a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = e0 + 32 * i + lane;
          a[i] = e < p.E ? p.offsets[e] : 0;
          b[i] = e < p.E ? p.offsets[e + 1] : 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = e0 + 32 * i + lane;
          falls |= b[i] < a[i];
          a[i] = min(max(a[i], 0), p.rows);
          b[i] = min(max(b[i], a[i]), p.rows);
          const uint32_t c = e < p.E ? units_of(b[i] - a[i]) : 0, scan = scan_of(c);
          if (e < p.E) {
            lo[e] = a[i];
            num[e] = b[i] - a[i];
            expert[e] = e;
            parts[e] = unit + scan - c;
          }
          dearest = max(dearest, cost_class<MODE, ROWS>(b[i] - a[i]));
          unit += __shfl_sync(ALL, scan, 31);
        }
      }
      dearest = __reduce_max_sync(ALL, dearest);
      if (lane == 0) {
        class_units[dearest] = unit;
        class_experts[dearest] = 1;
      }
    }
  } else {
    for (int e = threadIdx.x; e < p.E; e += THREADS) {
      falls |= p.offsets[e + 1] < p.offsets[e];
      const int a = min(max(p.offsets[e], 0), p.rows), b = min(max(p.offsets[e + 1], a), p.rows);
      lo[e] = a;
      num[e] = b - a;
      const int k = cost_class<MODE, ROWS>(b - a);
      atomicAdd(&class_units[k], units_of(b - a));
      atomicAdd(&class_experts[k], 1u);
    }
  }
  if (__syncthreads_or(falls)) {
    // Once more, in the experts' order: rows that an earlier expert has stay its own, so
    // that no two clusters write one row and a gradient counts it once.
    few = false;
    if (threadIdx.x < CLASSES) class_units[threadIdx.x] = class_experts[threadIdx.x] = 0;
    __syncthreads();
    if (warp == 0) {
      int taken = 0;  // behind the last row of the experts so far
      for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane, last = min(e, p.E - 1);
        const int from = min(max(p.offsets[last], 0), p.rows);
        const int to = min(max(p.offsets[last + 1], 0), p.rows);
        int most = to > from ? to : 0;  // of this lane's expert and those before
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
          const int o = __shfl_up_sync(ALL, most, i);
          if (lane >= i) most = max(most, o);
        }
        const int before = __shfl_up_sync(ALL, most, 1);
        const int a = max(from, max(taken, lane ? before : 0)), n = max(to - a, 0);
        if (e < p.E) {
          lo[e] = a;
          num[e] = n;
          atomicAdd(&class_units[cost_class<MODE, ROWS>(n)], units_of(n));
          atomicAdd(&class_experts[cost_class<MODE, ROWS>(n)], 1u);
        }
        taken = max(taken, __shfl_sync(ALL, most, 31));
      }
    }
    __syncthreads();
  }
  static_assert(THREADS / 32 >= CLASSES, "a warp a class");
  if (!few && warp < CLASSES) {
    uint32_t unit = 0, place = 0;
    for (int k = CLASSES - 1; k > warp; --k) {
      unit += class_units[k];
      place += class_experts[k];
    }
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const bool in = e < p.E && cost_class<MODE, ROWS>(num[e]) == warp;
      const uint32_t c = in ? units_of(num[e]) : 0;
      const uint32_t mask = __ballot_sync(ALL, in);
      if (!mask) continue;
      const uint32_t scan = scan_of(c);
      if (in) {
        const uint32_t at = place + __popc(mask & ((1u << lane) - 1));
        expert[at] = e;
        parts[at] = unit + scan - c;
      }
      place += __popc(mask);
      unit += __shfl_sync(ALL, scan, 31);
    }
  }
  uint32_t units = 0;
  int dearest = 0;
  for (int k = 0; k < CLASSES; ++k) {
    units += class_units[k];
    if (class_experts[k]) dearest = k;
  }
  // The ring: as many stages as fit with the rows of the largest tile there is.  What comes
  // from memory takes some 2 us from one stage's turn to its next, so that tiles of few rows
  // (one row each of 8 experts of 2048 x 1536: 18.7 us with 6 stages) need all they can get.
  units = same(units);
  dearest = same(dearest);
  const uint32_t b_bytes =
      MODE == GRADIENT ? S::B_BYTES : 2 * (dearest + 1) * (ROWS / 2 / CLASSES) * 128;
  const uint32_t stage_bytes = A_BYTES + b_bytes;
  const uint32_t stages = min(static_cast<uint32_t>(MAX_STAGES), S::RING_BYTES / stage_bytes);
  const Table table{parts, expert, lo, num};
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
  // One side's loads, by a warp of its own: a TMA instruction takes the warp that issues it
  // a hundred cycles and more, and a gather, whose operands differ from lane to lane, 60 a
  // lane.
  auto load = [&](auto which) {
    constexpr int side = decltype(which)::value;
    uint32_t it = 0, s = 0, ph = 1;  // stages armed and loaded; ring position, phase to wait for
    const bool stall = p.inject_stall && blockIdx.x == 0;  // test hook: stage 0 never fills
    const uint32_t fb0 = mapa_shared(full_bar(side, 0), 0);
    bool ok = true;
    int place = 0;
    for (uint32_t u = cluster; ok && u < units; u += clusters) {
      const Unit w = unit_at<MODE, ROWS>(u, p, table, place);
      const int kbs = same((w.sum + BK - 1) / BK), half = same(w.width / 2);
      const int expert = same(w.expert), sum0 = same(w.sum0), sum = same(w.sum);
      // this CTA's first feature, or row
      const int mine = same(side == 0 ? w.f0 + static_cast<int>(rank) * HALF
                                      : w.first + static_cast<int>(rank) * half);
      int32_t r[4];  // gather: this lane's four rows
      // Fours of rows that a CTA gathers: those with a row at all (what stands in the MMA's
      // other columns reaches no result; a gather of zeros takes as long as any).
      auto fours = [&](int of) { return (max(0, min(half, w.count - of * half)) + 3) / 4; };
      const int mine4 = same(fours(static_cast<int>(rank)));
      if constexpr (INDEXED && side == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = static_cast<int>(rank) * half + 4 * lane + i;
          const int row =
              at < w.count ? picked_row(p.gather[w.first + at], p.top, p.x_rows) : -1;
          r[i] = row >= 0 ? row : p.x_rows;
        }
      }
      for (int kb = 0; kb < kbs; ++kb, ++it) {
        if (!__all_sync(ALL, mbar_wait_bounded(empty_bar(s), ph, limit, &abort_flag))) {
          if (lane == 0) give_up(kErrTimeoutProducer);
          ok = false;
          break;
        }
        const uint32_t st = sbase + s * stage_bytes + side * A_BYTES, fb = fb0 + 8u * s;
        const int rows = min(BK, sum - kb * BK);  // gradient: positions of this stage,
        const int read = (rows + 15) & ~15;       // and those that the MMAs read
        constexpr int BOXES = side == 0 ? 2 : S::B_BYTES / BOX;  // gradient: of 64 features
        const uint32_t tx = MODE == GRADIENT ? BOXES * 128 * read
                            : side == 0      ? A_BYTES
                            : INDEXED        ? mine4 * 2 * 512
                                             : 2 * half * 128;
        auto arm = [&] {  // by one lane, the one that loads where one does
          stage_tx[side][s] = tx;
          if (leader) {
            const uint32_t tx1 = INDEXED && side == 1 ? fours(1) * 2 * 512 : tx;
            other_tx[side][s] = tx1;
            mbar_arrive_expect_tx(full_bar(side, s), tx + tx1);
          }
        };
        const bool load = !(stall && it == 0);
        if constexpr (MODE == GRADIENT) {
          const CUtensorMap* map = side == 0 ? maps.w : maps.x;
          const int pos = sum0 + kb * BK;
          if (rows == BK) {
            if (elect_one()) {
              arm();
              if (load) {
#pragma unroll
                for (int i = 0; i < BOXES; ++i)
                  tma_load_2d_pair(st + i * BOX, map + 3, fb, mine + 64 * i, pos);
              }
            }
          } else {
            // An expert's last rows: in boxes, and the last of sixteen by the gather,
            // which ends in zeros and not in the next expert's rows.
            const int whole = rows & ~15;
            if (elect_one()) {
              arm();
              if (load) {
#pragma unroll
                for (int g = 0; g < 3; ++g)
                  if (whole & (16 << g)) {
                    const int at = whole & ~((32 << g) - 1);  // behind the larger boxes
#pragma unroll
                    for (int i = 0; i < BOXES; ++i)
                      tma_load_2d_pair(st + i * BOX + at * 128, map + g, fb, mine + 64 * i,
                                       pos + at);
                  }
              }
            }
            __syncwarp();
            if (load && read > whole && lane < 4 * BOXES) {
              const int i = lane % BOXES, at = whole + 4 * (lane / BOXES);
#pragma unroll
              for (int j = 0; j < 4; ++j) r[j] = at + j < rows ? pos + at + j : p.rows;
              tma_gather4_pair(st + i * BOX + at * 128, side == 0 ? &maps.w1 : &maps.x1, fb,
                               mine + 64 * i, r);
            }
          }
        } else if constexpr (side == 0) {
          if (elect_one()) {
            arm();
            if (load) {
              if constexpr (MODE == PRODUCT) {
                tma_load_3d_pair(st, &maps.w[3], fb, mine, kb * BK, expert);
                tma_load_3d_pair(st + BOX, &maps.w[3], fb, mine + 64, kb * BK, expert);
              } else {
                tma_load_3d_pair(st, &maps.w[3], fb, kb * BK, mine, expert);
                tma_load_3d_pair(st + BOX, &maps.w[3], fb, kb * BK + 64, mine, expert);
              }
            }
          }
        } else if constexpr (INDEXED) {
          if (lane == 0) arm();
          __syncwarp();
          if (load && lane < mine4) {
            tma_gather4_pair(st + lane * 512, &maps.x1, fb, kb * BK, r);
            tma_gather4_pair(st + b_bytes / 2 + lane * 512, &maps.x1, fb, kb * BK + 64, r);
          }
        } else if (elect_one()) {
          arm();
          if (load) {
#pragma unroll
            for (int i = 3; i >= 0; --i)
              if (half & (16 << i)) {
                const int at = half & ~((32 << i) - 1);  // behind the larger boxes
                tma_load_2d_pair(st + at * 128, &maps.x[i], fb, kb * BK, mine + at);
                tma_load_2d_pair(st + b_bytes / 2 + at * 128, &maps.x[i], fb, kb * BK + 64,
                                 mine + at);
              }
          }
        }
        __syncwarp();
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (lane == 0) {
      // Both CTAs' loads complete in rank 0, which waits for all of them -- counting as
      // done what either CTA never issued -- before either may leave.
      volatile int never = 0;
      if (!leader) {
        for (uint32_t i = 0; i < stages; ++i)
          st_shared_cluster_u32(
              mapa_shared(smem_u32(const_cast<uint32_t*>(&peer_tx[side][i])), 0),
              stage_tx[side][i]);
        st_shared_cluster_u32(
            mapa_shared(smem_u32(const_cast<uint32_t*>(&peer_loaded[side])), 0), it);
        mbar_arrive_cluster(mapa_shared(peer_done_bar(side), 0));
      } else {
        uint32_t it1 = it;
        if (mbar_wait_bounded<true>(peer_done_bar(side), 0, 2 * limit, &never))
          it1 = peer_loaded[side];
        else
          atomicOr(p.status, kErrTimeoutDrain);
        const uint32_t hi = it > it1 ? it : it1;
        for (uint32_t i = hi > stages ? hi - stages : 0; i < hi; ++i) {
          const uint32_t si = i % stages, phi = (i / stages) & 1u;
          const bool armed = i < it, loaded0 = armed && !(stall && i == 0), loaded1 = i < it1;
          if (!armed) {
            mbar_arrive_expect_tx(full_bar(side, si), peer_tx[side][si]);
          } else {
            const uint32_t missing =
                (loaded0 ? 0u : stage_tx[side][si]) + (loaded1 ? 0u : other_tx[side][si]);
            if (missing) {  // once the MMA issuer has given up on the stage
              mbar_wait_bounded(full_bar(side, si), phi, 2 * limit, &abort_flag);
              mbar_complete_tx(full_bar(side, si), missing);
            }
          }
          if (!mbar_wait_bounded(full_bar(side, si), phi, limit, &never))
            atomicOr(p.status, kErrTimeoutDrain);
        }
      }
    }
    __syncwarp();
  };

  if (warp == 0) {
    load(std::integral_constant<int, 0>{});
  } else if (warp == 2 + EPI_WARPS) {
    load(std::integral_constant<int, 1>{});
  } else if (warp == 1) {
    if (leader) {
      uint32_t t = 0, s = 0, ph = 0;  // accumulators filled; ring position and its phase
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {  // a warp-uniform outcome
        return __all_sync(ALL, mbar_wait_bounded(bar, parity, limit, &abort_flag)) != 0;
      };
      int place = 0;
      auto both = [&](uint32_t s, uint32_t parity) {  // sides of a stage, asked for at once
        const bool a = mbar_try_wait(full_bar(0, s), parity), b = mbar_try_wait(full_bar(1, s), parity);
        return __all_sync(ALL, (a || mbar_wait_bounded(full_bar(0, s), parity, limit, &abort_flag)) &&
                                   (b || mbar_wait_bounded(full_bar(1, s), parity, limit, &abort_flag))) != 0;
      };
      for (uint32_t u = cluster; ok && u < units; u += clusters) {
        const Unit w = unit_at<MODE, ROWS>(u, p, table, place);
        const int sum = same(w.sum), kbs = (sum + BK - 1) / BK;
        const int tail = (sum - (kbs - 1) * BK + 15) / 16;  // MMAs of the last stage
        const uint32_t idesc =
            make_idesc(p.kind, MODE != TRANSPOSED, MODE == GRADIENT, TILE_F, same(w.width));
        // an accumulator whose last but one filling has been read
        auto next = [&] { return t < 2 || wait(released_bar(t & 1u), ((t - 2) >> 1) & 1u); };
        for (int kb = 0; kb < kbs; ++kb) {
          const int in = LONG ? kb % S::SEGMENT : kb;
          const bool last = kb + 1 == kbs || (LONG && in + 1 == S::SEGMENT);
          if ((in == 0 && !next()) || !both(s, ph)) {
            if (lane == 0) give_up(kErrTimeoutMma);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + (t & 1u) * ROWS;
          const uint32_t st = sbase + s * stage_bytes;
          const uint32_t a = desc_word(st, MODE == TRANSPOSED ? 16 : BOX);
          const uint32_t b = desc_word(st + A_BYTES, MODE == GRADIENT ? BOX : 16);
          // 16 of the sum: 32 bytes along a K-major row, of two halves; 16 rows of 128 bytes
          auto at_a = [&](int kk) -> uint32_t {
            return a + (MODE == TRANSPOSED ? kk / 4 * (BOX >> 4) + kk % 4 * 2 : kk * 128);
          };
          auto at_b = [&](int kk) -> uint32_t {
            return b + (MODE == GRADIENT ? kk * 128 : kk / 4 * (b_bytes >> 5) + kk % 4 * 2);
          };
          const uint32_t more = in > 0 ? 1u : 0u;
          const bool full = kb + 1 < kbs || tail == BK / 16;
          if (elect_one()) {
            if (full) {
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk)
                mma_pair(d, at_a(kk), at_b(kk), idesc, kk > 0 ? 1u : more);
            } else {
              for (int kk = 0; kk < tail; ++kk)
                mma_pair(d, at_a(kk), at_b(kk), idesc, kk > 0 ? 1u : more);
            }
            mma_commit_pair_multicast(empty_bar(s), 0x3);
            if (last) mma_commit_pair_multicast(acc_bar(t & 1u), 0x3);
          }
          __syncwarp();
          if (last) ++t;
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (kbs == 0) {  // (nothing to add up; the epilogue writes zeros)
          if (!next()) {
            if (lane == 0) give_up(kErrTimeoutMma);
            break;
          }
          if (elect_one()) mma_commit_pair_multicast(acc_bar(t & 1u), 0x3);
          __syncwarp();
          ++t;
        }
      }
      if (elect_one()) mma_commit_pair(drain_bar);
      __syncwarp();
      volatile int never = 0;
      if (!mbar_wait_bounded(drain_bar, 0, limit, &never) && lane == 0)
        atomicOr(p.status, kErrTimeoutDrain);
    } else {
      uint32_t t = 0;
      bool ok = true;
      int place = 0;
      for (uint32_t u = cluster; ok && u < units; u += clusters) {
        const int kbs = (unit_at<MODE, ROWS>(u, p, table, place).sum + BK - 1) / BK;
        const int fillings = LONG ? max(1, (kbs + S::SEGMENT - 1) / S::SEGMENT) : 1;
        for (int i = 0; i < fillings; ++i, ++t) {
          ok = __all_sync(ALL, mbar_wait_bounded(read_bar(t & 1u), (t >> 1) & 1u, limit,
                                                 &abort_flag, 64));
          if (!ok) {
            if (lane == 0) give_up(kErrTimeoutEpilogue);
            break;
          }
          if (lane == 0) mbar_arrive_cluster(mapa_shared(released_bar(t & 1u), 0));
          __syncwarp();
        }
      }
    }
    __syncwarp();
  } else {
    // two warps a lane quarter, every other 32 columns each
    const int q = warp & 3, odd = (warp - 2) >> 2;
    // A 16-bit gradient's rows of 128 bytes take the space of two warps: the first of a
    // quarter's two does them all (all do where TMA cannot write them).
    const bool alone = MODE == GRADIENT && !LONG && p.out_tma;
    const uint32_t piece =
        sbase + S::RING_BYTES + (warp - 2) * S::PIECE_BYTES * (alone ? 2 : 1);
    uint32_t t = 0;
    bool ok = true;
    int place = 0;
    for (uint32_t u = cluster; ok && u < units; u += clusters) {
      const Unit w = unit_at<MODE, ROWS>(u, p, table, place);
      const int kbs = (w.sum + BK - 1) / BK;
      const int fillings = LONG ? max(1, (kbs + S::SEGMENT - 1) / S::SEGMENT) : 1;
      const int feature = w.f0 + static_cast<int>(rank) * HALF + q * 32 + lane;
      constexpr int HELD = LONG ? ROWS / 64 : 1;
      float held[HELD][32];
      for (int i = 0; i < fillings; ++i, ++t) {
        const uint32_t b = t & 1u;
        if (!__all_sync(ALL,
                        mbar_wait_bounded(acc_bar(b), (t >> 1) & 1u, limit, &abort_flag, 64))) {
          if (lane == 0) give_up(kErrTimeoutEpilogue);
          __syncwarp();
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + b * ROWS;
        auto release = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(leader ? released_bar(b) : read_bar(b));
        };
        if constexpr (LONG) {
#pragma unroll
          for (int c = 0; c < HELD; ++c) {
            const int at = (2 * c + odd) * 32;
            if (at < w.count) {
              uint32_t r[32];
              tmem_ld_32cols(taddr + at, r);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float v = w.sum ? __uint_as_float(r[j]) : 0.f;
                held[c][j] = i ? held[c][j] + v : v;
              }
            }
          }
          release();
          if (i + 1 == fillings) {
#pragma unroll
            for (int c = 0; c < HELD; ++c) {
              const int at = (2 * c + odd) * 32;
              if (at < w.count) {
                auto& v = reinterpret_cast<uint32_t(&)[32]>(held[c]);
                if constexpr (MODE == GRADIENT)
                  store_rows(v, p, &maps.out, piece, w.expert, feature - lane, w.first + at, lane);
                else
                  store_chunk<true>(v, p, &maps.out, piece, w, at, feature, lane);
              }
            }
          }
        } else if constexpr (MODE == GRADIENT) {
          // 32 columns from `at` on in 16 words (no terms: the accumulator was not written)
          auto packed = [&](int at, auto& v, auto from) {
            uint32_t r[32];
            tmem_ld_32cols(taddr + at, r);
            tmem_ld_wait();
            auto pack = [&](auto dtype) {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                v[decltype(from)::value + j] =
                    w.sum ? pack16<decltype(dtype)::value>(r[2 * j], r[2 * j + 1]) : 0u;
            };
            if (p.out_dtype == MHR_BF16)
              pack(std::integral_constant<int, MHR_BF16>{});
            else
              pack(std::integral_constant<int, MHR_F16>{});
          };
          const int row = feature - lane;
          if (alone) {
            if (odd) release();
#pragma unroll 1
            for (int at = 0; !odd && at < w.count; at += 64) {
              uint32_t v[32];
              packed(at, v, std::integral_constant<int, 0>{});
              packed(at + 32, v, std::integral_constant<int, 16>{});
              if (at + 64 >= w.count) release();
              store_rows(v, p, &maps.out, piece, w.expert, row, w.first + at, lane);
            }
          } else {
            if (32 * odd >= w.count) release();
#pragma unroll 1
            for (int at = 32 * odd; at < w.count; at += 64) {
              uint32_t v[16];
              packed(at, v, std::integral_constant<int, 0>{});
              if (at + 64 >= w.count) release();
#pragma unroll
              for (int k = 0; k < 4; ++k)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 piece + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4)),
                             "r"(v[4 * k]), "r"(v[4 * k + 1]), "r"(v[4 * k + 2]), "r"(v[4 * k + 3])
                             : "memory");
              __syncwarp();
              const int col = w.first + at;
              store_ragged(static_cast<uint16_t*>(p.out) + w.expert * p.stride_o + row * p.ldo + col,
                           p.ldo, min(32, p.K - row), min(32, p.N - col), piece, lane);
              __syncwarp();
            }
          }
        } else {
          if (32 * odd >= w.count) release();
#pragma unroll 1
          for (int at = 32 * odd; at < w.count; at += 64) {
            uint32_t r[32];
            tmem_ld_32cols(taddr + at, r);
            tmem_ld_wait();
            if (w.sum == 0) {  // no terms: the accumulator was not written
#pragma unroll
              for (int j = 0; j < 32; ++j) r[j] = 0;
            }
            if (at + 64 >= w.count) release();
            store_chunk<false>(r, p, &maps.out, piece, w, at, feature, lane);
          }
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the pair's MMAs or arrivals may touch it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, S::TMEM_COLS);
  }
}

// Rows as TMA reads them, into scratch with a pitch of whole 16 bytes: of the parts
// (experts) that have rows of tokens where `offsets` is given, or those that `index`
// over `top` picks (zeros where it picks none).  A warp takes a row.
template <typename Word>
__global__ void __launch_bounds__(256)
    rows_kernel(const uint16_t* src, int64_t src_rows, int64_t cols, int64_t ld, int64_t stride,
                const int32_t* offsets, const int32_t* index, int top, uint16_t* dst,
                int64_t rows, int64_t dst_ld) {
  grid_dependency_wait();
  const int64_t part = blockIdx.y;
  if (offsets && offsets[part + 1] <= offsets[part]) return;
  src += part * stride;
  dst += part * rows * dst_ld;
  constexpr int EACH = sizeof(Word) / 2, DEEP = sizeof(Word) == 16 ? 4 : 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t words = cols / EACH;  // (a whole number)
  for (int64_t q = static_cast<int64_t>(blockIdx.x) * 8 + warp; q < rows; q += gridDim.x * 8) {
    const int64_t r = index ? picked_row(index[q], top, static_cast<int>(src_rows)) : q;
    const Word* from = reinterpret_cast<const Word*>(src + r * ld);
    Word* to = reinterpret_cast<Word*>(dst + q * dst_ld);
    for (int64_t c = lane; c < words; c += 32 * DEEP) {
      Word v[DEEP];
#pragma unroll
      for (int i = 0; i < DEEP; ++i) {
        v[i] = Word{};
        if (r >= 0 && c + 32 * i < words) v[i] = from[c + 32 * i];
      }
#pragma unroll
      for (int i = 0; i < DEEP; ++i)
        if (c + 32 * i < words) to[c + 32 * i] = v[i];
    }
  }
}

template <int MODE, bool INDEXED, bool LONG>
cudaError_t launch_t(const Maps& m, const Params& p, cudaLaunchConfig_t cfg) {
  using S = Shape<LONG>;
  auto kern = routed_pair_kernel<MODE, INDEXED, LONG>;
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = S::SMEM;
  static int most[64];  // by device; under the library's lock
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  int clusters = device < 64 ? most[device] : 0;
  if (!clusters) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM)) !=
        cudaSuccess)
      return e;
    cfg.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg)) != cudaSuccess) return e;
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    if (device < 64) most[device] = clusters;
  }
  // As many units as there can be at most: every row tile but one of an expert's full.
  const int64_t tiles = MODE == GRADIENT
                            ? static_cast<int64_t>(p.E) * p.n_tiles
                            : (p.rows < p.E ? p.rows : p.E) + p.rows / S::ROWS;
  const int64_t units = tiles * p.f_tiles;
  if (units > 0x3fffffff) return cudaErrorInvalidConfiguration;
  if (units < clusters) clusters = static_cast<int>(units);
  cfg.gridDim = dim3(2 * clusters);
  cfg.numAttrs = 2;
  char name[64];
  snprintf(name, sizeof(name), "routed_pair_kernel<%s%s%s>",
           MODE == GRADIENT ? "gradient" : MODE == TRANSPOSED ? "transposed" : "product",
           INDEXED ? ",indexed" : "", LONG ? ",long" : "");
  note_main_kernel(name, 2 * clusters, static_cast<int>(units));
  e = cudaLaunchKernelEx(&cfg, kern, m, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int64_t operand_bytes(const void* p, int64_t parts, int64_t rows, int64_t cols, int64_t ld,
                      int64_t stride, int64_t picked) {
  if (rows == 0 || cols == 0 ||
      (picked == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows == 1 || ld % 8 == 0) &&
       (parts == 1 || stride % 8 == 0)))
    return 0;
  int64_t n;
  if (__builtin_mul_overflow(picked ? picked : parts * rows, (cols + 7) / 8 * 16, &n) ||
      n > INT64_MAX - 255)
    return -1;
  return (n + 255) / 256 * 256;
}

cudaError_t ready(const void* p, int64_t parts, int64_t rows, int64_t cols, int64_t ld,
                  int64_t stride, const int32_t* offsets, const int32_t* index, int64_t top,
                  int64_t picked, char** scratch, cudaStream_t s, Operand* out) {
  const int64_t bytes = operand_bytes(p, parts, rows, cols, ld, stride, index ? picked : 0);
  if (bytes == 0) {
    *out = {p, rows, ld, stride};
    return cudaSuccess;
  }
  const int64_t dst_ld = (cols + 7) / 8 * 8, dst_rows = index ? picked : rows;
  uint16_t* dst = reinterpret_cast<uint16_t*>(*scratch);
  *out = {dst, dst_rows, dst_ld, dst_rows * dst_ld};
  *scratch += bytes;
  const int64_t blocks = (dst_rows + 7) / 8;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096),
                     static_cast<unsigned>(parts));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool vectors = reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0 &&
                       stride % 8 == 0 && cols % 8 == 0;
  auto kern = vectors ? rows_kernel<uint4> : rows_kernel<uint16_t>;
  note_launch();
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, kern, static_cast<const uint16_t*>(p), rows, cols, ld, stride,
                         offsets, index, static_cast<int>(top), dst, dst_rows, dst_ld);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_product(const ProductArgs& a, void* scratch, const DeviceCtl& ctl,
                           cudaStream_t s) {
  const bool gradient = a.kind == ProductKind::gradient;
  Params p = {};
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
  const bool wide = a.out_dtype == MHR_F32;
  const int tile_rows = wide ? 128 : 256;
  p.f_tiles = static_cast<int32_t>(((gradient ? a.K : a.N) + TILE_F - 1) / TILE_F);
  p.n_tiles = static_cast<int32_t>((a.N + tile_rows - 1) / tile_rows);
  p.kind = a.dtype == MHR_BF16 ? 1 : 0;
  p.out_dtype = a.out_dtype;
  p.pairs = !wide && reinterpret_cast<uintptr_t>(a.out) % 4 == 0 && a.ldo % 2 == 0 &&
            (!gradient || a.stride_o % 2 == 0);
  // (TMA clips a box at the row's end in whole 16 bytes only)
  const int64_t per = wide ? 4 : 8, out_rows = gradient ? a.K : a.out_rows;
  p.out_tma = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.N % per == 0 &&
              (out_rows == 1 || a.ldo % per == 0) &&
              (!gradient || a.E == 1 || a.stride_o % per == 0) && (gradient || !a.scatter);
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
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.gridDim = dim3(2 * (ctl.sm_count / 2));

  Maps m = {};
  const auto type = a.dtype == MHR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const auto swizzle = CU_TENSOR_MAP_SWIZZLE_128B;
  if (p.out_tma) {
    const int64_t size = wide ? 4 : 2, parts = gradient ? a.E : 1;
    const int64_t ld = out_rows == 1 ? a.N : a.ldo;
    const uint64_t dims[3] = {static_cast<uint64_t>(a.N), static_cast<uint64_t>(out_rows),
                              static_cast<uint64_t>(parts)};
    const uint64_t pitch[2] = {static_cast<uint64_t>(ld * size),
                               static_cast<uint64_t>((parts == 1 ? out_rows * ld : a.stride_o) * size)};
    const uint32_t box[3] = {gradient && !wide ? 64u : 32u, 32, 1};
    if (encode_tmap_3d(&m.out,
                       wide ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                       a.out, dims, pitch, box,
                       gradient ? swizzle : CU_TENSOR_MAP_SWIZZLE_NONE) != CUDA_SUCCESS)
      p.out_tma = 0;  // (a pitch past TMA's: the rows go out from registers)
  }
  if (!none) {
    char* at = static_cast<char*>(scratch);
    Operand x, w;
    const bool in_order = a.gather && (gradient || a.rows > FEW_ROWS);
    cudaError_t e = ready(a.x, 1, a.x_rows, a.K, a.ldx, 0, nullptr, in_order ? a.gather : nullptr,
                          a.top, a.rows, &at, s, &x);
    if (e != cudaSuccess) return e;
    if (in_order) p.gather = nullptr;
    auto rows_map = [&](CUtensorMap* map, const Operand& r, int64_t cols, uint32_t box) {
      // (one row has no pitch of its own to go by)
      const int64_t ld = r.rows == 1 ? (cols + 7) / 8 * 8 : r.ld;
      return encode_tmap_2d(map, type, r.p, cols, r.rows, ld * 2, 64, box, swizzle) ==
             CUDA_SUCCESS;
    };
    bool ok = true;
    if (gradient) {
      e = ready(a.w, 1, a.out_rows, a.N, a.ldw, 0, nullptr, a.scatter, 1, a.rows, &at, s, &w);
      if (e != cudaSuccess) return e;
      p.scatter = nullptr;
      for (int i = 0; i < 4; ++i)
        ok = ok && rows_map(&m.w[i], x, a.K, 16u << i) && rows_map(&m.x[i], w, a.N, 16u << i);
      ok = ok && rows_map(&m.w1, x, a.K, 1) && rows_map(&m.x1, w, a.N, 1);
    } else {
      const bool t = a.kind == ProductKind::transposed;
      const int64_t rows = t ? a.N : a.K, cols = t ? a.K : a.N;
      e = ready(a.w, a.E, rows, cols, a.ldw, a.stride_w, a.offsets, nullptr, 1, 0, &at, s, &w);
      if (e != cudaSuccess) return e;
      const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows),
                                static_cast<uint64_t>(a.E)};
      const int64_t ld = rows == 1 ? (cols + 7) / 8 * 8 : w.ld;
      const int64_t stride = a.E == 1 ? rows * ((cols + 7) / 8 * 8) : w.stride;
      const uint64_t pitch[2] = {static_cast<uint64_t>(ld) * 2, static_cast<uint64_t>(stride) * 2};
      const uint32_t box[3] = {64, 128, 1};
      ok = encode_tmap_3d(&m.w[3], type, w.p, dims, pitch, box, swizzle) == CUDA_SUCCESS;
      for (int i = 0; i < 4; ++i) ok = ok && rows_map(&m.x[i], x, a.K, 16u << i);
      ok = ok && rows_map(&m.x1, x, a.K, 1);
    }
    if (!ok) return cudaErrorInvalidValue;
  }
  MainKernelEvents ev(s);
  auto by_width = [&](auto mode, auto indexed) {
    constexpr int MODE = decltype(mode)::value;
    constexpr bool INDEXED = decltype(indexed)::value;
    return wide ? launch_t<MODE, INDEXED, true>(m, p, cfg) : launch_t<MODE, INDEXED, false>(m, p, cfg);
  };
  auto by_index = [&](auto mode) {
    return p.gather ? by_width(mode, std::true_type{}) : by_width(mode, std::false_type{});
  };
  switch (a.kind) {
    case ProductKind::gradient:
      return by_width(std::integral_constant<int, GRADIENT>{}, std::false_type{});
    case ProductKind::transposed: return by_index(std::integral_constant<int, TRANSPOSED>{});
    default: return by_index(std::integral_constant<int, PRODUCT>{});
  }
}

}  // namespace routed
}  // namespace mhr
