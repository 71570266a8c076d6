// Low-rank adapters of many requests (gemm_routed_adapters):
//   out_t = y_t + scale_a (x_t down_a^T) up_a,   a = which[t].
//
// Few rows: a cluster of 8 CTAs takes a row.  Each CTA sums its eighth of x against
// down_a's rows, the r sums of all eight meet in every CTA's shared memory, and each
// writes its eighth of the output: one launch, and every byte of the adapter is read
// once, by a CTA of its own.
//
// Many rows: rows are sorted by adapter (routed_sort.cu), and a cluster takes 128 of
// one adapter on tcgen05.  Its CTAs split x's columns for v = x down^T, add up their
// parts through distributed shared memory, and split the output's columns for v up.
// Few rows are bound by latency (one of 4096 x 4096, rank 16: 4.4 us; 48 of 4096 x 11008:
// 7), many by HBM in phases, x, v's exchange, y (8192 of 4096 x 4096, rank 64: 62 us, 3.3
// TB/s; 17 of it the exchange, the sort and the launches).
// v stays in 32 bits on the way: for the tensor cores it is written as a sum of 16-bit
// terms (three of bf16, two of fp16), good to 2^-22 of a row's largest, whatever the
// result's type: a row's value does not go by how many rows come with it.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "mhr_gemm.h"
#include "mhr_mxfp4.h"
#include "mxfp4_common.cuh"
#include "routed_internal.h"

namespace mhr {
namespace routed {
namespace {

using mx::elect_one;
using mx::from_float;
using mx::to_float;

constexpr uint32_t ALL = 0xffffffffu;

struct AdapterParams {
  const void *x, *down, *up, *y;
  void* out;
  const int32_t* which;
  const float* scales;
  int64_t ldx, ldd, stride_d, ldu, stride_u, ldy, ldo;
  int32_t T, K, N, L, rank;
};

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 floats(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
};
template <>
struct Pair<__half> {
  static __device__ __forceinline__ float2 floats(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
};
template <typename T>
__device__ __forceinline__ void floats8(const uint4& w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = Pair<T>::floats(u[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

// n elements by `threads` threads, 16 bytes and four loads at a time where both ends allow.
template <typename O>
__device__ __forceinline__ void copy_row(O* to, const O* from, int n, int thread, int threads) {
  constexpr int PER = 16 / sizeof(O);
  int done = 0;
  if (((reinterpret_cast<uintptr_t>(to) | reinterpret_cast<uintptr_t>(from)) & 15u) == 0) {
    const int words = n / PER;
    const uint4* src = reinterpret_cast<const uint4*>(from);
    uint4* dst = reinterpret_cast<uint4*>(to);
    for (int c = thread; c < words; c += 4 * threads) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i * threads < words) v[i] = src[c + i * threads];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i * threads < words) dst[c + i * threads] = v[i];
    }
    done = words * PER;
  }
  for (int c = done + thread; c < n; c += 4 * threads) {
    O v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i * threads < n) v[i] = from[c + i * threads];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i * threads < n) to[c + i * threads] = v[i];
  }
}

// ------------------------------------------------------------------ few rows

constexpr int CTAS = 8;
constexpr int ROW_THREADS = 256;
constexpr int ROW_WARPS = ROW_THREADS / 32;

// VEC: x, the adapters, y and out in vectors of 8 columns (aligned, K and N multiples
// of 8); else element by element.
template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(ROW_THREADS) __cluster_dims__(CTAS, 1, 1)
    adapters_row_kernel(const AdapterParams p) {
  __shared__ float part[CTAS][MAX_RANK];  // every CTA's sums
  __shared__ float v[MAX_RANK];
  __shared__ float sums[ROW_THREADS * 8];
  const int t = blockIdx.x / CTAS, rank = blockIdx.x % CTAS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  const int a = p.which[t];
  const bool some = a >= 0 && a < p.L;
  constexpr int W = VEC ? 8 : 1;
  const O* y = static_cast<const O*>(p.y) + t * p.ldy;
  O* out = static_cast<O*>(p.out) + t * p.ldo;
  const int n_each = ((p.N + CTAS - 1) / CTAS + 7) & ~7;
  const int n0 = min(p.N, rank * n_each), n1 = min(p.N, n0 + n_each);
  if (!some) {  // (the whole cluster)
    if (static_cast<const void*>(y) != out)
      copy_row(out + n0, y + n0, n1 - n0, threadIdx.x, ROW_THREADS);
    return;
  }
  // (every CTA has to run before another writes its shared memory)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const T* x = static_cast<const T*>(p.x) + t * p.ldx;
  const T* down = static_cast<const T*>(p.down) + a * p.stride_d;
  const int k_each = ((p.K + CTAS - 1) / CTAS + 7) & ~7;
  const int k0 = min(p.K, rank * k_each), k1 = min(p.K, k0 + k_each);
  constexpr int G = 4;  // rows of down a warp takes at once
  bool first = true;
  for (int j0 = warp * G; j0 < p.rank; j0 += ROW_WARPS * G) {
    float acc[G] = {};
    for (int k = k0 + lane * W; k < k1; k += 32 * W) {
      if constexpr (VEC) {
        const uint4 xw = *reinterpret_cast<const uint4*>(x + k);
        uint4 dw[G];
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (j0 + g < p.rank)
            dw[g] = *reinterpret_cast<const uint4*>(down + (j0 + g) * p.ldd + k);
        float xf[8];
        floats8<T>(xw, xf);
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (j0 + g < p.rank) {
            float df[8];
            floats8<T>(dw[g], df);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[g] = fmaf(xf[i], df[i], acc[g]);
          }
      } else {
        const float xf = to_float(x[k]);
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (j0 + g < p.rank) acc[g] = fmaf(xf, to_float(down[(j0 + g) * p.ldd + k]), acc[g]);
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int m = 16; m; m >>= 1) acc[g] += __shfl_xor_sync(ALL, acc[g], m);
    if (first) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    first = false;
    // lane 8 g' + c sends row g' of the group to CTA c: every lane has a CTA of the cluster
    static_assert(CTAS == 8 && G * CTAS == 32, "a lane for each row and CTA");
    const int g = lane >> 3;
    float mine = acc[0];
#pragma unroll
    for (int i = 1; i < G; ++i) mine = g == i ? acc[i] : mine;
    if (j0 + g < p.rank)
      st_shared_cluster_u32(mapa_shared(smem_u32(&part[rank][j0 + g]), lane & 7),
                            __float_as_uint(mine));
  }
  if (first) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  cluster_sync_all();
  for (int j = threadIdx.x; j < p.rank; j += ROW_THREADS) {
    float s = 0;
#pragma unroll
    for (int c = 0; c < CTAS; ++c) s += part[c][j];
    v[j] = (p.scales ? p.scales[a] : 1.f) * s;
  }
  __syncthreads();
  const T* up = static_cast<const T*>(p.up) + a * p.stride_u;
  const int cols = (n1 - n0 + W - 1) / W;               // vectors of columns
  const int groups = cols ? max(1, min(ROW_THREADS / cols, p.rank)) : 1;  // that share a column's rows
  if (groups > 1) {
    const int c = threadIdx.x % cols, g = threadIdx.x / cols;
    float acc[W] = {};
    if (g < groups)
      for (int j = g; j < p.rank; j += groups) {
        const T* at = up + j * p.ldu + n0 + c * W;
        if constexpr (VEC) {
          float f[8];
          floats8<T>(*reinterpret_cast<const uint4*>(at), f);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = fmaf(v[j], f[i], acc[i]);
        } else {
          acc[0] = fmaf(v[j], to_float(*at), acc[0]);
        }
      }
    if (g < groups)
#pragma unroll
      for (int i = 0; i < W; ++i) sums[(g * cols + c) * W + i] = acc[i];
    __syncthreads();
    for (int n = threadIdx.x; n < n1 - n0; n += ROW_THREADS) {
      float s = 0;
      for (int g2 = 0; g2 < groups; ++g2) s += sums[g2 * cols * W + n];
      out[n0 + n] = from_float<O>(to_float(y[n0 + n]) + s);
    }
  } else {
    for (int c = threadIdx.x; c < cols; c += ROW_THREADS) {
      float acc[W] = {};
      for (int j = 0; j < p.rank; ++j) {
        const T* at = up + j * p.ldu + n0 + c * W;
        if constexpr (VEC) {
          float f[8];
          floats8<T>(*reinterpret_cast<const uint4*>(at), f);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = fmaf(v[j], f[i], acc[i]);
        } else {
          acc[0] = fmaf(v[j], to_float(*at), acc[0]);
        }
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int n = n0 + c * W + i;
        out[n] = from_float<O>(to_float(y[n]) + acc[i]);
      }
    }
  }
}

// ------------------------------------------------------------------ many rows

// Tiles: 128 rows of one adapter, in the order of routed_sort.cu.
constexpr int TILE = 128;
// Of x's columns a stage: two boxes of 128 bytes a row, since a stage costs the warps that
// load and multiply some 700 cycles whatever it holds (513 rows of 4096 x 4096 and rank 64
// 36.5 us with one box, 34.6 with two; 4096 x 11008 and rank 16 47.4 and 43.5).
constexpr int BK = 128;
constexpr int XBOX = TILE * 128;
constexpr int BLOCK_N = 128;                  // of the output's columns an accumulator
constexpr int EPI_WARPS = 8;
constexpr int EPI_THREADS = 32 * EPI_WARPS;
constexpr int TILE_THREADS = 64 + EPI_THREADS;  // warp 0 loads, 1 multiplies, 2-9 the rest
constexpr int SLOT = 32 * 128;                // 32 rows of y and of the output, 128 bytes each
constexpr int MAX_STAGES = 8;
constexpr uint32_t TMEM_COLS = 512, ACC0 = 256;  // v's sums up to column 256, then the output's

struct TileMaps {
  CUtensorMap x, x32, x1, down, up, y, y1, out;  // x and y: whole boxes, and single rows
};

struct TileParams {
  const int32_t *offsets, *order;
  const float* scales;
  const void* y;
  void* out;
  int64_t ldy, ldo;
  int32_t T, K, N, L, rank;
  int32_t pad;          // rank, in steps of 16
  int32_t stages, slots;  // of `up` and of y; x and `down` have the memory of both first
  int32_t stages1;
  int32_t kind, copy;   // 0 fp16, 1 bf16; copy: rows without an adapter are copied
  int32_t rows_tma;     // y and the output can go by TMA
  uint32_t* status;
  uint64_t wait_limit_ns;
  int32_t inject_stall;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t x, const int32_t (&r)[4]) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]),
      "r"(r[3])
      : "memory");
}
// mma_f16 by the low words of the descriptors: the address and the leading offset.
__device__ __forceinline__ uint32_t desc_word(uint32_t saddr, uint32_t lbo_bytes) {
  return ((saddr & 0x3FFFFu) >> 4) | (lbo_bytes >> 4) << 16;
}
__device__ __forceinline__ void mma_words(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(mx::DESC_HI_SW128)
      : "memory");
}
__device__ __forceinline__ float4 ld_shared_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_u4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (std::is_same_v<T, __half>) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// A tile: 128 sorted rows from `first` on, `count` of them, of adapter `a` (L: of none).
struct Tile {
  int a, first, count;
};

// T: of x and the adapters; O: of y and the output.  BOXES: 64 columns of v each.
//
// v is given to the tensor cores as TERMS values of T whose sum it is to 2^-24 of it (three
// of bf16) or 2^-22 of the row's largest (two of fp16, taken times a power of two a row so
// that neither leaves fp16's range).
template <typename T, typename O, int BOXES>
__global__ void __launch_bounds__(TILE_THREADS, 1)
    adapters_tile_kernel(const __grid_constant__ TileMaps maps, const TileParams p) {
  constexpr bool HALF = std::is_same_v<T, __half>, WIDE = sizeof(O) == 4;
  constexpr int TERMS = HALF ? 2 : 3;
  constexpr int SUMS = 4 / BOXES;              // accumulators of v (see below)
  constexpr int BOX_COLS = WIDE ? 32 : 64;     // of the output, 128 bytes
  constexpr int PARTS = 64 / BOX_COLS;         // boxes of a warp's half of a block
  extern __shared__ uint8_t smem_raw[];
  __shared__ alignas(8) uint64_t bars[4 * MAX_STAGES + 7 + 3 * EPI_WARPS];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ Tile tile_slot;
  __shared__ uint32_t scan_sums[TILE_THREADS / 32];
  __shared__ int32_t rows[TILE];
  __shared__ float row_max[2][HALF ? TILE : 1], row_unit[HALF ? TILE : 1];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };        // of x and `down`
  auto empty_bar = [&](int s) { return bar0 + 8u * (MAX_STAGES + s); };
  auto up_bar = [&](int s) { return bar0 + 8u * (2 * MAX_STAGES + s); };
  auto up_free_bar = [&](int s) { return bar0 + 8u * (3 * MAX_STAGES + s); };
  auto acc_bar = [&](int b) { return bar0 + 8u * (4 * MAX_STAGES + b); };
  auto free_bar = [&](int b) { return bar0 + 8u * (4 * MAX_STAGES + 2 + b); };
  const uint32_t sums_bar = bar0 + 8u * (4 * MAX_STAGES + 4);
  const uint32_t v_bar = bar0 + 8u * (4 * MAX_STAGES + 5);
  const uint32_t drain_bar = bar0 + 8u * (4 * MAX_STAGES + 6);
  auto y_bar = [&](int w, int s) { return bar0 + 8u * (4 * MAX_STAGES + 7 + 3 * w + s); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  int ctas;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
  const int tile_no = blockIdx.x / ctas;

  grid_dependency_wait();
  // Which tile: the bins' tiles, summed up.  (Bin L holds the rows without an adapter.)
  if (threadIdx.x == 0) tile_slot = {-1, 0, 0};
  __syncthreads();
  int base = 0;
  for (int b0 = 0; b0 <= p.L && base <= tile_no; b0 += TILE_THREADS) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    int lo = 0, n = 0;
    if (b <= p.L) {
      lo = p.offsets[b];
      n = (b < p.L ? p.offsets[b + 1] : p.T) - lo;
    }
    const int tiles = b == p.L && !p.copy ? 0 : (n + TILE - 1) / TILE;
    int scan = tiles;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const int o = __shfl_up_sync(ALL, scan, i);
      if (lane >= i) scan += o;
    }
    if (lane == 31) scan_sums[warp] = scan;
    __syncthreads();
    int lower = base, all = 0;
    for (int i = 0; i < TILE_THREADS / 32; ++i) {
      if (i < warp) lower += scan_sums[i];
      all += scan_sums[i];
    }
    const int at = tile_no - (lower + scan - tiles);
    if (at >= 0 && at < tiles) tile_slot = {b, lo + at * TILE, min(TILE, n - at * TILE)};
    base += all;
    __syncthreads();
  }
  const Tile tile = tile_slot;
  if (tile.a < 0) return;  // (the whole cluster: there are fewer tiles)
  // This CTA's stages of x's columns, and its blocks of the output's.
  const int kbs = (p.K + BK - 1) / BK, blocks = (p.N + BLOCK_N - 1) / BLOCK_N;
  const int kb0 = kbs * rank / ctas, kb1 = kbs * (rank + 1) / ctas;
  const int n0 = blocks * rank / ctas, n1 = blocks * (rank + 1) / ctas;
  for (int i = threadIdx.x; i < TILE; i += TILE_THREADS)
    rows[i] = i < tile.count ? p.order[tile.first + i] : -1;
  __syncthreads();
  if (tile.a == p.L) {  // copied: a warp a row
    const int c0 = n0 * BLOCK_N, c1 = min(p.N, n1 * BLOCK_N);
    for (int i = warp; i < tile.count; i += TILE_THREADS / 32) {
      const O* from = static_cast<const O*>(p.y) + rows[i] * p.ldy;
      O* to = static_cast<O*>(p.out) + rows[i] * p.ldo;
      copy_row(to + c0, from + c0, c1 - c0, lane, 32);
    }
    return;
  }

  const int v_cols = p.pad;
  const uint32_t stage_bytes = TILE * 128 + BOXES * 64 * 128;
  const uint32_t v_base = smem_u32(smem);  // v's parts, then its terms
  const uint32_t v_bytes = max(TERMS * BOXES * TILE * 128, TILE * (BOXES * 64 * 4 + 16));
  const uint32_t ring = v_base + ((v_bytes + 1023) & ~1023u);
  const uint32_t slots = ring + p.stages * stage_bytes;
  if (threadIdx.x == 0) {
    for (int s = 0; s < MAX_STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(up_bar(s), 1);
      mbar_init(up_free_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_bar(b), 1);
      mbar_init(free_bar(b), EPI_WARPS);
    }
    mbar_init(sums_bar, 1);
    mbar_init(v_bar, EPI_THREADS);
    mbar_init(drain_bar, 1);
    for (int w = 0; w < EPI_WARPS; ++w)
      for (int s = 0; s < 3; ++s) mbar_init(y_bar(w, s), 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint64_t limit = p.wait_limit_ns;
  auto wait = [&](uint32_t bar, uint32_t parity, uint32_t sleep = 0) {  // by a whole warp
    return __all_sync(ALL, mbar_wait_bounded(bar, parity, limit, &abort_flag, sleep)) != 0;
  };
  auto give_up = [&](uint32_t bit) {
    if (lane == 0) {
      if (!abort_flag) atomicOr(p.status, bit);
      abort_flag = 1;
    }
    __syncwarp();
  };
  // v's sums go on in the next of SUMS accumulators every `run` stages: the tensor cores add by
  // truncation, which takes 1.4e-8 of a sum off with its first 16 terms and 3e-7 after 256.
  // (One accumulator was no faster: 8192 rows of 4096 x 4096 and rank 64 62 us either way.)
  const int run = max(1, (kb1 - kb0 + SUMS - 1) / SUMS);

  if (warp == 0) {
    // Rows 32 by 32: a box where they lie together (else gathered, by the epilogue's warps).
    int from[4];
    bool lying[4], whole = true;  // whole: one box of all
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      from[g] = __shfl_sync(ALL, rows[g * 32], 0);
      lying[g] = __all_sync(ALL, rows[g * 32 + lane] < 0 || rows[g * 32 + lane] == from[g] + lane) &&
                 from[g] >= 0;
      whole &= lying[g] ? from[g] == from[0] + 32 * g : tile.count <= 32 * g;
    }
    const int a = __shfl_sync(ALL, tile.a, 0);
    const bool stall = p.inject_stall && blockIdx.x == 0;
    uint32_t s = 0, ph = 1, it = 0, up_it = 0;
    bool ok = true;
    const uint32_t tx1 = 2 * (XBOX + v_cols * 128), tx2 = 2 * v_cols * 128;
    auto next = [&](uint32_t empty) {
      ok = wait(empty, ph);
      if (!ok) give_up(kErrTimeoutProducer);
      return ok;
    };
    auto advance = [&](uint32_t of) {
      __syncwarp();
      if (++s == of) {
        s = 0;
        ph ^= 1u;
      }
    };
    for (int kb = kb0; ok && kb < kb1; ++kb) {
      if (!next(empty_bar(s))) break;
      const uint32_t st = ring + s * 2 * stage_bytes, fb = full_bar(s);
      if (elect_one()) {
        mbar_arrive_expect_tx(fb, tx1);
        if (!(stall && kb == kb0)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // (a second box past K comes as zeros)
            const int k = kb * BK + 64 * h;
            if (whole) {
              tma_load_2d(st + h * XBOX, &maps.x, fb, k, from[0]);
            } else {
#pragma unroll
              for (int g = 0; g < 4; ++g)
                if (lying[g]) tma_load_2d(st + h * XBOX + g * 4096, &maps.x32, fb, k, from[g]);
            }
            tma_load_3d(st + 2 * XBOX + h * v_cols * 128, &maps.down, fb, k, 0, a);
          }
        }
      }
      ++it;
      advance(p.stages1);
    }
    // The memory of x and `down` goes to `up` and y when v's sums are there.
    s = 0;
    ph = 1;
    if (kb1 > kb0 && ok && !wait(sums_bar, 0)) {
      give_up(kErrTimeoutProducer);
      ok = false;
    }
    auto load_up = [&](int n) {
      if (!next(up_free_bar(s))) return;
      const uint32_t st = ring + s * stage_bytes, fb = up_bar(s);
      if (elect_one()) {
        mbar_arrive_expect_tx(fb, tx2);
        if (!(stall && kb0 == kb1 && n == n0)) {
          tma_load_3d(st, &maps.up, fb, n * BLOCK_N, 0, a);
          tma_load_3d(st + v_cols * 128, &maps.up, fb, n * BLOCK_N + 64, 0, a);
        }
      }
      ++up_it;
      advance(p.stages);
    };
    int n = n0;
    for (; ok && n < n1 && n < n0 + p.stages; ++n) load_up(n);
    cluster_sync_all();
    cluster_arrive();
    cluster_wait();
    for (; ok && n < n1; ++n) load_up(n);
    if (lane == 0) {  // what is still on its way, before the CTA may leave
      volatile int never = 0;
      auto drain = [&](auto bar, uint32_t of, uint32_t n, bool stalled, uint32_t tx) {
        for (uint32_t i = n > of ? n - of : 0; i < n; ++i) {
          if (stalled && i == 0) {
            mbar_wait_bounded(bar(0), 0, 2 * limit, &abort_flag);
            mbar_complete_tx(bar(0), tx);
          }
          if (!mbar_wait_bounded(bar(i % of), (i / of) & 1u, limit, &never))
            atomicOr(p.status, kErrTimeoutDrain);
        }
      };
      drain(full_bar, p.stages1, it, stall, tx1);
      drain(up_bar, p.stages, up_it, stall && kb0 == kb1, tx2);
    }
    __syncwarp();
  } else if (warp == 1) {
    uint32_t s = 0, ph = 0;
    bool ok = true;
    auto advance = [&](uint32_t of) {
      __syncwarp();
      if (++s == of) {
        s = 0;
        ph ^= 1u;
      }
    };
    const uint32_t id1 = make_idesc(p.kind, false, false, TILE, v_cols);
    const uint32_t id2 = make_idesc(p.kind, false, true, TILE, BLOCK_N);
    int in = 0;           // stages that v's present accumulator has
    uint32_t d = tmem;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!wait(full_bar(s), ph)) {
        give_up(kErrTimeoutMma);
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t st = ring + s * 2 * stage_bytes;
      if (in == run) {
        in = 0;
        d += BOXES * 64;
      }
      const uint32_t a = desc_word(st, 16), b = desc_word(st + 2 * XBOX, 16);
      const uint32_t more = in > 0 ? 1u : 0u;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          mma_words(d, a + kk / 4 * (XBOX >> 4) + kk % 4 * 2, b + kk / 4 * (v_cols * 8) + kk % 4 * 2,
                    id1, kk > 0 ? 1u : more);
        mma_commit(empty_bar(s));
        if (kb + 1 == kb1) mma_commit(sums_bar);
      }
      ++in;
      advance(p.stages1);
    }
    s = ph = 0;
    cluster_sync_all();
    cluster_arrive();
    cluster_wait();
    if (ok && n1 > n0 && !wait(v_bar, 0)) {
      give_up(kErrTimeoutMma);
      ok = false;
    }
    for (int n = n0; ok && n < n1; ++n) {
      const int t = n - n0, b = t & 1;
      if ((t >= 2 && !wait(free_bar(b), ((t - 2) >> 1) & 1u)) || !wait(up_bar(s), ph)) {
        give_up(kErrTimeoutMma);
        break;
      }
      tc_fence_after();
      const uint32_t st = ring + s * stage_bytes;
      const uint32_t v0 = desc_word(v_base, 16), up0 = desc_word(st, v_cols * 128);
      if (elect_one()) {
        for (int kk = 0; kk < v_cols / 16; ++kk)
#pragma unroll
          for (int term = 0; term < TERMS; ++term)
            mma_words(tmem + ACC0 + b * BLOCK_N,
                      v0 + (term * BOXES + kk / 4) * (TILE * 8) + kk % 4 * 2, up0 + kk * 128, id2,
                      kk > 0 || term > 0 ? 1u : 0u);
        mma_commit(up_free_bar(s));
        mma_commit(acc_bar(b));
      }
      advance(p.stages);
    }
    if (elect_one()) mma_commit(drain_bar);
    __syncwarp();
    volatile int never = 0;
    if (!mbar_wait_bounded(drain_bar, 0, limit, &never) && lane == 0)
      atomicOr(p.status, kErrTimeoutDrain);
    __syncwarp();
  } else {
    // Warp e: lane quarter q, half h of the columns.
    const int e = warp - 2, q = warp & 3, h = e >> 2;
    const int row = q * 32 + lane;  // of the tile
    const int mine = rows[row];
    const int first = rows[q * 32], n_rows = max(0, min(32, tile.count - q * 32));
    const bool lie = __all_sync(ALL, lane >= n_rows || mine == first + lane);
    const bool load = p.rows_tma && n_rows > 0;      // y by TMA, in a box or gathered; the
    const bool store = load && lie && n_rows == 32;  // output in a box that is all of it
    int32_t four[4];  // of a gather: rows 4 lane .. 4 lane + 3 of this warp's
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = __shfl_sync(ALL, mine, (4 * lane + i) & 31);
      four[i] = r >= 0 ? r : p.T;
    }
    const uint32_t slot0 = slots + e * p.slots * SLOT;
    const int boxes = n_rows > 0 ? (n1 - n0) * PARTS : 0;
    auto box_col = [&](int i) {
      return (n0 + i / PARTS) * BLOCK_N + h * 64 + i % PARTS * BOX_COLS;
    };
    int fetched = 0, done = 0;
    // y's box i into its slot
    auto fetch = [&](int i) {
      const uint32_t slot = slot0 + i % p.slots * SLOT;
      const int col = box_col(i);
      if (load) {
        fetched = i + 1;  // (columns past N, of the last block, come as zeros)
        const uint32_t bar = y_bar(e, i % p.slots);
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, SLOT);
          if (lie) tma_load_2d(slot, &maps.y, bar, col, first);
        }
        __syncwarp();
        if (!lie && lane < 8) tma_gather4(slot + lane * 512, &maps.y1, bar, col, four);
      }
    };
    bool ok = true;
    // x's rows that lie in no box of 32: four gathers a warp, of 16 rows.  (An operand that
    // differs from lane to lane makes a TMA instruction some 60 cycles of the warp's; all
    // by the loading warp, a stage took 1160 cycles and more.)
    {
      const int g = e >> 1, r0 = g * 32, of = rows[r0];
      const bool box = of >= 0 && __all_sync(ALL, rows[r0 + lane] < 0 || rows[r0 + lane] == of + lane);
      bool whole = rows[0] >= 0;  // (one box has them all)
      for (int k = 0; k < TILE; k += 32)
        whole &= __all_sync(ALL, rows[k + lane] < 0 || rows[k + lane] == rows[0] + k + lane) != 0;
      if (!whole && !box) {
        int32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = rows[(r0 + (e & 1) * 16 + 4 * lane + i) & (TILE - 1)];
          r[i] = at >= 0 ? at : p.T;
        }
        const bool stall = p.inject_stall && blockIdx.x == 0;
        uint32_t s = 0, ph = 1;
        for (int i = 0; i < kb1 - kb0; ++i) {
          if (!wait(empty_bar(s), ph)) {
            give_up(kErrTimeoutProducer);
            ok = false;
            break;
          }
          if (lane < 4 && !(stall && i == 0)) {
            const uint32_t to = ring + s * 2 * stage_bytes + (r0 + (e & 1) * 16) * 128 + lane * 512;
            tma_gather4(to, &maps.x1, full_bar(s), (kb0 + i) * BK, r);
            tma_gather4(to + XBOX, &maps.x1, full_bar(s), (kb0 + i) * BK + 64, r);
          }
          __syncwarp();
          if (++s == static_cast<uint32_t>(p.stages1)) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
    // v: this thread's half of its row's columns, summed over accumulators and CTAs.
    constexpr int COLS = BOXES * 32;
    const int half_cols = v_cols / 2;  // (a multiple of 8)
    if (kb1 > kb0) {
      ok = ok && wait(sums_bar, 0, 128);
      if (!ok) give_up(kErrTimeoutEpilogue);
      tc_fence_after();
    }
    // (the slots have been x's until now)
    for (int i = 0; ok && i < min(boxes, p.slots - 1); ++i) fetch(i);
    const uint32_t pitch = BOXES * 64 * 4 + 16;
    const uint32_t part = v_base + row * pitch + h * half_cols * 4;
    const int used = kb1 > kb0 ? (kb1 - kb0 + run - 1) / run : 0;
    float v[COLS] = {};
#pragma unroll
    for (int k = 0; k < SUMS; ++k) {
      if (ok && k < used) {
        uint32_t d[COLS / 8][8];
        const uint32_t at =
            tmem + (static_cast<uint32_t>(q * 32) << 16) + k * (BOXES * 64) + h * half_cols;
#pragma unroll
        for (int c = 0; c < COLS; c += 8)
          if (c < half_cols) mx::tmem_ld_8cols(at + c, d[c / 8]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < COLS; ++c)
          if (c < half_cols) v[c] += __uint_as_float(d[c / 8][c % 8]);
      }
    }
    if (ctas > 1) {
#pragma unroll
      for (int c = 0; c < COLS; c += 4)
        if (c < half_cols)
          st_shared_v4(part + c * 4, make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]));
    }
    cluster_sync_all();
    const float scale = p.scales ? p.scales[tile.a] : 1.f;
    uint32_t terms[TERMS][COLS / 2];
    float high = 0;
    {
      // The others' parts, a CTA's at once: 32 KB of 64 columns, which take some 2000 cycles
      // to come.
      for (int i = 1; i < ctas; ++i) {
        const uint32_t from = mapa_shared(part, (rank + i) % ctas);
        float4 o[COLS / 4];
#pragma unroll
        for (int c = 0; c < COLS; c += 4)
          if (c < half_cols) o[c / 4] = ld_shared_cluster_v4(from + c * 4);
#pragma unroll
        for (int c = 0; c < COLS; c += 4)
          if (c < half_cols) {
            v[c] += o[c / 4].x;
            v[c + 1] += o[c / 4].y;
            v[c + 2] += o[c / 4].z;
            v[c + 3] += o[c / 4].w;
          }
      }
      // (v's columns past the rank are x times down's missing rows: an infinity there would be
      // NaN, and reach every column of the output by up's)
#pragma unroll
      for (int c = 0; c < COLS; ++c) v[c] = h * half_cols + c < p.rank ? v[c] * scale : 0.f;
      cluster_arrive();  // this thread has read the parts
      float unit = 1.f;
      if constexpr (HALF) {
        // A power of two a row that brings its largest finite value to [2^13, 2^14).
#pragma unroll
        for (int c = 0; c < COLS; ++c) high = fmaxf(high, isfinite(v[c]) ? fabsf(v[c]) : 0.f);
        row_max[h][row] = high;
        asm volatile("barrier.cta.sync 1, %0;" ::"n"(EPI_THREADS) : "memory");
        high = fmaxf(row_max[0][row], row_max[1][row]);
        const int x = static_cast<int>(__float_as_uint(high) >> 23);  // 0: below 2^-126
        if (high > 0.f) {
          const int up = min(13 + 127 - x, 126);  // (-114 at least: both powers are normal)
          unit = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
          if (h == 0) row_unit[row] = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
        } else if (h == 0) {
          row_unit[row] = 1.f;
        }
      }
#pragma unroll
      for (int c = 0; c < COLS; c += 2) {
        float a = v[c] * unit, b = v[c + 1] * unit;
#pragma unroll
        for (int k = 0; k < TERMS; ++k) {
          const uint32_t w = pack2<T>(a, b);
          terms[k][c / 2] = w;
          const float2 f = Pair<T>::floats(w);
          // (what is infinite has no rest)
          a = isfinite(f.x) ? a - f.x : 0.f;
          b = isfinite(f.y) ? b - f.y : 0.f;
        }
      }
    }
    cluster_wait();  // all have: the terms take the parts' place
#pragma unroll
    for (int k = 0; k < TERMS; ++k)
#pragma unroll
      for (int c = 0; c < COLS; c += 8)
        if (c < half_cols) {
          const int col = h * half_cols + c, box = col / 64, chunk = col % 64 / 8;
          st_shared_u4(v_base + (k * BOXES + box) * (TILE * 128) + row * 128 +
                           ((chunk ^ (row & 7)) << 4),
                       make_uint4(terms[k][c / 2], terms[k][c / 2 + 1], terms[k][c / 2 + 2],
                                  terms[k][c / 2 + 3]));
        }
    fence_proxy_async_smem();
    mbar_arrive(v_bar);
    if constexpr (HALF)  // (row_unit)
      asm volatile("barrier.cta.sync 1, %0;" ::"n"(EPI_THREADS) : "memory");
    const float unit = HALF ? row_unit[row] : 1.f;

    // Element by element over a box's rows, 16 of a lane's at a time: first all the loads.
    auto for_elements = [&](const auto& get, const auto& put, int col) {
      constexpr int EACH = BOX_COLS / 32;
      for (int j0 = 0; j0 < n_rows; j0 += 16 / EACH) {
        O v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int j = j0 + k / EACH, c = lane + k % EACH * 32;
          v[k] = get(min(j, n_rows - 1), c, j * 128 + ((c * sizeof(O)) ^ ((j & 7) << 4)),
                     j < n_rows && col + c < p.N);
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int j = j0 + k / EACH, c = lane + k % EACH * 32;
          put(min(j, n_rows - 1), c, j * 128 + ((c * sizeof(O)) ^ ((j & 7) << 4)),
              j < n_rows && col + c < p.N, v[k]);
        }
      }
    };
    const int total = (n1 - n0) * PARTS;
    for (int i = 0; i < total; ++i) {
      const int t = i / PARTS, b = t & 1;
      if (ok && i % PARTS == 0 && !wait(acc_bar(b), (t >> 1) & 1u, 64)) {
        give_up(kErrTimeoutEpilogue);
        ok = false;
      }
      if (!ok) break;
      const int col = box_col(i);
      const uint32_t slot = slot0 + i % p.slots * SLOT;
      const bool work = n_rows > 0 && col < p.N;
      if (load) {
        if (!wait(y_bar(e, i % p.slots), (i / p.slots) & 1u)) {
          give_up(kErrTimeoutEpilogue);
          ok = false;
          break;
        }
        done = i + 1;
      } else if (work) {  // rows that TMA cannot read
        for_elements([&](int j, int c, uint32_t at, bool in) {
          O v = O{};
          if (in) v = static_cast<const O*>(p.y)[rows[q * 32 + j] * p.ldy + col + c];
          return v;
        }, [&](int, int, uint32_t at, bool, O v) {
          if constexpr (WIDE)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(slot + at), "r"(__float_as_uint(v)) : "memory");
          else
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(slot + at),
                         "h"(*reinterpret_cast<uint16_t*>(&v))
                         : "memory");
        }, col);
        __syncwarp();
      }
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + ACC0 + b * BLOCK_N +
                           h * 64 + i % PARTS * BOX_COLS;
      uint32_t d[BOX_COLS / 32][32];
#pragma unroll
      for (int k = 0; k < BOX_COLS / 32; ++k) tmem_ld_32cols(acc + 32 * k, d[k]);
      tmem_ld_wait();
      if (i % PARTS == PARTS - 1) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(free_bar(b));
      }
      if (work) {
        const uint32_t line = slot + lane * 128;
#pragma unroll
        for (int k = 0; k < 8; ++k) {  // 16 bytes of the row
          const uint32_t at = line + ((k ^ (lane & 7)) << 4);
          uint4 w = ld_shared_u4(at);
          uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (WIDE) {
              const float o = __uint_as_float(d[0][4 * k + j]) * unit;
              u[j] = __float_as_uint(__uint_as_float(u[j]) + o);
            } else {
              const int c = 8 * k + 2 * j;
              const float2 f = Pair<O>::floats(u[j]);
              u[j] = pack2<O>(fmaf(__uint_as_float(d[c / 32][c % 32]), unit, f.x),
                              fmaf(__uint_as_float(d[c / 32][c % 32 + 1]), unit, f.y));
            }
          }
          st_shared_u4(at, make_uint4(u[0], u[1], u[2], u[3]));
        }
        if (store) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tma_store_2d(&maps.out, slot, col, first);
        } else {
          __syncwarp();
          if (load) {  // eight lanes a row of 128 bytes
            constexpr int PER = 16 / sizeof(O);
            const int c = lane & 7, left = p.N - (col + c * PER);
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int j = 4 * k + (lane >> 3);
              v[k] = ld_shared_u4(slot + j * 128 + ((c ^ (j & 7)) << 4));
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int j = 4 * k + (lane >> 3);
              // (N is whole 16 bytes)
              if (j < n_rows && left > 0)
                *reinterpret_cast<uint4*>(static_cast<O*>(p.out) + rows[q * 32 + j] * p.ldo + col +
                                          c * PER) = v[k];
            }
          } else {
            for_elements([&](int, int, uint32_t at, bool) {
              O v;
              if constexpr (WIDE) {
                uint32_t u;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(u) : "r"(slot + at) : "memory");
                v = __uint_as_float(u);
              } else {
                uint16_t u;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(slot + at) : "memory");
                v = *reinterpret_cast<O*>(&u);
              }
              return v;
            }, [&](int j, int c, uint32_t, bool in, O v) {
              if (in) static_cast<O*>(p.out)[rows[q * 32 + j] * p.ldo + col + c] = v;
            }, col);
          }
          __syncwarp();
          // (what is read and written here, before TMA's next load of the slot)
          if (load) fence_proxy_async_smem();
        }
      }
      if (lane == 0) bulk_commit_group();
      // The slot of the box before this one: its store has had a box's time to read it.
      if (i + p.slots - 1 < boxes) {
        if (lane == 0) bulk_wait_group_read<1>();
        __syncwarp();
        fetch(i + p.slots - 1);
      }
    }
    if (lane == 0) {
      bulk_wait_group<0>();
      if (load) {  // fetched and not waited for, where a wait has run out
        volatile int never = 0;
        for (; done < fetched; ++done)
          mbar_wait_bounded(y_bar(e, done % p.slots), (done / p.slots) & 1u, limit, &never);
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

bool aligned(const void* p, int64_t elements) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && elements % 8 == 0;
}

template <typename T, typename O>
cudaError_t launch_rows(const AdapterArgs& a, const AdapterParams& p, cudaStream_t s) {
  const bool vec = aligned(a.x, a.T == 1 ? 0 : a.ldx) && aligned(a.down, a.ldd) &&
                   a.stride_d % 8 == 0 && aligned(a.up, a.ldu) && a.stride_u % 8 == 0 &&
                   a.K % 8 == 0 && a.N % 8 == 0;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.T * CTAS));
  cfg.blockDim = dim3(ROW_THREADS);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_launch();
  const cudaError_t e = vec ? cudaLaunchKernelEx(&cfg, adapters_row_kernel<T, O, true>, p)
                            : cudaLaunchKernelEx(&cfg, adapters_row_kernel<T, O, false>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_out(const AdapterArgs& a, const AdapterParams& p, cudaStream_t s) {
  if (a.out_dtype == MHR_F32) return launch_rows<T, float>(a, p, s);
  if (a.out_dtype == MHR_BF16) return launch_rows<T, __nv_bfloat16>(a, p, s);
  return launch_rows<T, __half>(a, p, s);
}

template <typename T, typename O, int BOXES>
cudaError_t launch_tiles(const AdapterArgs& a, const AdapterParams& r, TileParams p,
                         const TileMaps& maps, const DeviceCtl& ctl, cudaStream_t s) {
  auto kern = adapters_tile_kernel<T, O, BOXES>;
  constexpr bool HALF = std::is_same_v<T, __half>;
  constexpr int TERMS = HALF ? 2 : 3;
  constexpr int STAGE = TILE * 128 + BOXES * 64 * 128;
  constexpr int TERM_BYTES = TERMS * BOXES * TILE * 128, PART_BYTES = TILE * (BOXES * 64 * 4 + 16);
  constexpr int V = ((TERM_BYTES > PART_BYTES ? TERM_BYTES : PART_BYTES) + 1023) / 1024 * 1024;
  constexpr int MOST = HALF ? 222 * 1024 : 224 * 1024;
  constexpr int SLOTS = (MOST - V - 3 * EPI_WARPS * SLOT) / STAGE >= 2 ? 3 : 2;
  constexpr int FIT = (MOST - V - SLOTS * EPI_WARPS * SLOT) / STAGE;
  constexpr int STAGES = FIT < MAX_STAGES ? FIT : MAX_STAGES;
  static_assert(STAGES >= 2, "shared memory");
  constexpr int SMEM = V + STAGES * STAGE + SLOTS * EPI_WARPS * SLOT + 1024;
  p.stages = STAGES;
  constexpr int STAGES1 = (STAGES * STAGE + SLOTS * EPI_WARPS * SLOT) / (2 * STAGE);
  static_assert(STAGES1 >= 2, "shared memory");
  p.stages1 = STAGES1 < MAX_STAGES ? STAGES1 : MAX_STAGES;
  p.slots = SLOTS;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  // CTAs a tile: as many as leave every tile room to run at once.  Clusters of 8 do not
  // pack into all of the SMs (2048 rows of 4096 x 4096, rank 16, as 16 of them: 43 us, as
  // clusters of 4: 30), so they stay below half; and every CTA more sends the others
  // 128 x rank sums, which pays only against long rows (256 rows, 8 CTAs / 4: rank 16, K + N
  // of 15104 30 / 42 us, 8192 22 / 26, 2048 17 / 16; rank 64, 8192 38 / 33, 1024 32 / 21).
  // Where the adapters may make tiles for more than two rounds of 8, they are 4 as well
  // (1024 rows of 4096 x 11008 with 64 adapters in no order: 167 / 93 us).
  const int64_t full = (a.T + TILE - 1) / TILE;
  // every bin's tiles but one are full
  const int64_t tiles = a.T / TILE + (a.T < a.L + 1 ? a.T : a.L + 1);
  const bool wide = full * 16 <= ctl.sm_count && tiles * 4 <= ctl.sm_count &&
                    a.K + a.N >= 256 * a.rank;
  int ctas = wide ? 8 : 4;
  while (ctas > 1 && full * ctas > ctl.sm_count) ctas /= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * ctas));
  cfg.blockDim = dim3(TILE_THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  note_main_kernel("adapters_tile_kernel", static_cast<int>(tiles * ctas), static_cast<int>(tiles));
  e = cudaLaunchKernelEx(&cfg, kern, maps, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// Whether every row has a cluster of its own.  That kernel's time grows with the rows, the
// tiles' hardly does until they fill the device.  In us (bf16, 8 adapters), rows' / tiles':
//     K, N, rank       128 rows    256 rows    512 rows
//     4096, 4096, 16    9.2 / 22   17.0 / 21   30.5 / 22
//     4096, 4096, 64   17.0 / 34   29.8 / 32   62   / 33
//     1024, 1024, 16    7.0 / 15   13.1 / 15   23.3 / 16
//     4096, 11008, 16  13.4 / 32   25.3 / 30   55   / 31
// Up to 512 rows that may have an adapter for every 8 of them keep to rows too: with 64
// adapters in no order, a tile each, the last line's 512 rows are 57 / 100.  How many of
// them are in use is not known here: with 4 of the 64, a run of rows each, 54 / 44.
bool by_rows(const AdapterArgs& a) { return a.T <= 256 || (a.T <= 512 && a.T <= 8 * a.L); }

cudaError_t launch_many(const AdapterArgs& a, const AdapterParams& r, void* scratch,
                        const DeviceCtl& ctl, cudaStream_t s) {
  char* at = static_cast<char*>(scratch);
  int32_t* offsets = reinterpret_cast<int32_t*>(at);
  at += align256(4 * (a.L + 1));
  int32_t* order = reinterpret_cast<int32_t*>(at);
  at += align256(4 * a.T);
  cudaError_t e = launch_sort(a.which, a.T, a.L, offsets, order, s);
  if (e != cudaSuccess) return e;
  Operand x{}, down{}, up{};
  if (a.K > 0) {
    e = ready(a.x, 1, a.T, a.K, a.ldx, 0, nullptr, nullptr, 1, 0, &at, s, &x);
    if (e != cudaSuccess) return e;
    e = ready(a.down, a.L, a.rank, a.K, a.ldd, a.stride_d, offsets, nullptr, 1, 0, &at, s, &down);
    if (e != cudaSuccess) return e;
  }
  e = ready(a.up, a.L, a.rank, a.N, a.ldu, a.stride_u, offsets, nullptr, 1, 0, &at, s, &up);
  if (e != cudaSuccess) return e;

  TileParams p = {};
  p.offsets = offsets;
  p.order = order;
  p.scales = a.scales;
  p.y = a.y;
  p.out = a.out;
  p.ldy = a.ldy;
  p.ldo = a.ldo;
  p.T = r.T;
  p.K = r.K;
  p.N = r.N;
  p.L = r.L;
  p.rank = r.rank;
  p.pad = (r.rank + 15) / 16 * 16;
  p.kind = a.dtype == MHR_BF16 ? 1 : 0;
  p.copy = a.y != a.out;
  p.status = ctl.status;
  p.wait_limit_ns = ctl.wait_limit_ns;
  p.inject_stall = ctl.inject_stall;
  const int64_t size = a.out_dtype == MHR_F32 ? 4 : 2;
  auto rows_of_16 = [&](const void* q, int64_t ld) {
    return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld * size % 16 == 0;
  };
  // (TMA clips a box at the row's end in whole 16 bytes only)
  p.rows_tma = rows_of_16(a.y, a.ldy) && rows_of_16(a.out, a.ldo) && a.N * size % 16 == 0;
  TileMaps m = {};
  const auto type = a.dtype == MHR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const auto swizzle = CU_TENSOR_MAP_SWIZZLE_128B;
  auto parts = [&](CUtensorMap* map, const Operand& o, int64_t cols) {
    const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(a.rank),
                              static_cast<uint64_t>(a.L)};
    const int64_t ld = a.rank == 1 ? (cols + 7) / 8 * 8 : o.ld;
    const int64_t stride = a.L == 1 ? a.rank * ((cols + 7) / 8 * 8) : o.stride;
    const uint64_t pitch[2] = {static_cast<uint64_t>(ld) * 2, static_cast<uint64_t>(stride) * 2};
    const uint32_t box[3] = {64, static_cast<uint32_t>(p.pad), 1};
    return encode_tmap_3d(map, type, o.p, dims, pitch, box, swizzle) == CUDA_SUCCESS;
  };
  bool ok = parts(&m.up, up, a.N);
  if (a.K > 0) {
    for (CUtensorMap* map : {&m.x, &m.x32, &m.x1})
      ok = ok && encode_tmap_2d(map, type, x.p, a.K, a.T, x.ld * 2, 64,
                                map == &m.x ? TILE : map == &m.x32 ? 32 : 1,
                                swizzle) == CUDA_SUCCESS;
    ok = ok && parts(&m.down, down, a.K);
  }
  if (p.rows_tma) {
    const auto out_type = a.out_dtype == MHR_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint32_t cols = static_cast<uint32_t>(128 / size);
    // (a pitch past TMA's: rows one by one)
    p.rows_tma = encode_tmap_2d(&m.y, out_type, a.y, a.N, a.T, a.ldy * size, cols, 32, swizzle) ==
                     CUDA_SUCCESS &&
                 encode_tmap_2d(&m.y1, out_type, a.y, a.N, a.T, a.ldy * size, cols, 1, swizzle) ==
                     CUDA_SUCCESS &&
                 encode_tmap_2d(&m.out, out_type, a.out, a.N, a.T, a.ldo * size, cols, 32,
                                swizzle) == CUDA_SUCCESS;
  }
  if (!ok) return cudaErrorInvalidValue;
  MainKernelEvents ev(s);
  auto by_rank = [&](auto t, auto o) {
    using T = decltype(t);
    using O = decltype(o);
    return p.pad <= 64 ? launch_tiles<T, O, 1>(a, r, p, m, ctl, s)
                       : launch_tiles<T, O, 2>(a, r, p, m, ctl, s);
  };
  auto by_out = [&](auto t) {
    if (a.out_dtype == MHR_F32) return by_rank(t, float{});
    if (a.out_dtype == MHR_BF16) return by_rank(t, __nv_bfloat16{});
    return by_rank(t, __half{});
  };
  return a.dtype == MHR_BF16 ? by_out(__nv_bfloat16{}) : by_out(__half{});
}

}  // namespace

int64_t adapters_scratch(const AdapterArgs& a) {
  if (by_rows(a)) return 0;
  const int64_t each[3] = {
      a.K > 0 ? operand_bytes(a.x, 1, a.T, a.K, a.ldx, 0, 0) : 0,
      a.K > 0 ? operand_bytes(a.down, a.L, a.rank, a.K, a.ldd, a.stride_d, 0) : 0,
      operand_bytes(a.up, a.L, a.rank, a.N, a.ldu, a.stride_u, 0)};
  int64_t n = align256(4 * (a.L + 1)) + align256(4 * a.T);
  for (const int64_t b : each)
    if (b < 0 || __builtin_add_overflow(n, b, &n)) return -1;
  return n;
}

cudaError_t launch_adapters(const AdapterArgs& a, void* scratch, const DeviceCtl& ctl,
                            cudaStream_t s) {
  AdapterParams p;
  p.x = a.x;
  p.down = a.down;
  p.up = a.up;
  p.y = a.y;
  p.out = a.out;
  p.which = a.which;
  p.scales = a.scales;
  p.ldx = a.ldx;
  p.ldd = a.ldd;
  p.stride_d = a.stride_d;
  p.ldu = a.ldu;
  p.stride_u = a.stride_u;
  p.ldy = a.ldy;
  p.ldo = a.ldo;
  p.T = static_cast<int32_t>(a.T);
  p.K = static_cast<int32_t>(a.K);
  p.N = static_cast<int32_t>(a.N);
  p.L = static_cast<int32_t>(a.L);
  p.rank = static_cast<int32_t>(a.rank);
  if (!by_rows(a)) return launch_many(a, p, scratch, ctl, s);
  return a.dtype == MHR_BF16 ? launch_out<__nv_bfloat16>(a, p, s) : launch_out<__half>(a, p, s);
}

}  // namespace routed
}  // namespace mhr
