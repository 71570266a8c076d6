// The 4-bit product for few rows of A: C^T tiles of 128 columns of C (rows of
// B^T) x up to 128 rows of A, one CTA each, with the K blocks of a tile split
// over a cluster of CTAs when tiles are few.
//
// With few rows of A the product is a pass over B: N K 17/32 bytes against
// M N K multiply-adds.  So B takes the MMA's 128-row side, whole K-tiles of it
// stream in by TMA, and A's rows are the MMA's N (8 to 128 in steps of 8).
// The cluster's CTAs each hold a partial sum in TMEM; they meet in distributed
// shared memory and are added in rank order, so a result is the same from call
// to call.
//
// A plain A of few rows is quantised on the way by the CTA's other warps, each CTA
// its part of K, where that is little work (every tile of columns repeats it): one
// launch instead of two, and no packed A in memory.
//
// Bound by HBM, or by its latency where B is small.  GB300, packed A, weights out of
// cache: 24 x 11008 x 4096 8.8 us (2.8 TB/s), 32 x 28672 x 4096 13.7 (4.7 TB/s), 1 x
// 4096 x 4096 5.6; an empty launch of clusters takes 2.1 of them.  (The stage's MMAs
// are issued unrolled: with loops of a count known at run time only, a stage took 20 %
// longer.)
#include <type_traits>

#include "mhr_gemm.h"
#include "mhr_mxfp4.h"
#include "mxfp4_common.cuh"

namespace mhr {
namespace mx {
namespace {

constexpr int BK_BYTES = 128;         // 256 columns of K a stage: one swizzle row
constexpr int W_ROWS = 128;           // rows of B^T a tile: the MMA's M
constexpr int W_BYTES = W_ROWS * BK_BYTES;
constexpr int SF_BYTES = 1024;        // two scale tiles of 128 rows
constexpr int MAX_STAGES = 10;
constexpr int MAX_NT = 128;           // rows of A a tile: the MMA's N
constexpr int THREADS = 192;           // packed A
constexpr int PLAIN_THREADS = 512;     // A quantised here
constexpr int PLAIN_ROWS = 32;
// Rows x stages of K that a CTA quantises at most.  GB300, quantised here against by
// a kernel before: 1 x 4096 x 4096 (3 of them) 5.9 / 7.0 us, 8 x 11008 x 4096 (48)
// 9.5 / 10.0, 12 x 11008 x 4096 (72) 10.5 / 10.3, 24 x 11008 x 4096 (144) 13.6 / 10.7.
constexpr int PLAIN_TASKS = 50;
constexpr int PLAIN_BYTES = 32 * 1024;  // of the quantised part of A
constexpr int MAX_SPLIT = 8;
constexpr int SMEM_LIMIT = 227 * 1024;
constexpr uint32_t TMEM_COLS = 256;     // so that two CTAs fit an SM
constexpr int PAIR_NT = 32;             // up to this many rows two CTAs share an SM

struct NarrowParams {
  int32_t M, N;
  int32_t nt;              // rows of A a tile, a multiple of 8
  int32_t tiles_n, split;  // tiles along N; CTAs (K parts) a tile
  int32_t num_kb;          // stages of 256 columns in K
  int32_t blocks, kt;      // blocks of 32 in K; scale tiles a row
  int32_t stages, stage_bytes;
  uint32_t sf_col;         // TMEM: the accumulator, then 16 columns of scales a stage
  int32_t early_b;         // B is not written by the kernel before this one
  const void* a;           // plain A, its pitch, and whether its rows take 16-byte loads
  int64_t lda;
  int32_t K, vec_a;
  int32_t a_bytes;         // shared memory of its quantised part, before the ring
  const uint8_t* sfa;
  const uint8_t* sfb;
  void* C;
  int64_t ldc;
  int32_t c_dtype, vec_c;  // vec_c: 4 columns of C from a multiple of 4 on may be stored at once
  uint32_t* status;
  uint64_t wait_limit_ns;
  int32_t inject_stall;
};

__device__ __forceinline__ void store_c(const NarrowParams& p, int64_t at, float v) {
  if (p.c_dtype == MHR_F32)
    static_cast<float*>(p.C)[at] = v;
  else if (p.c_dtype == MHR_BF16)
    static_cast<__nv_bfloat16*>(p.C)[at] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p.C)[at] = __float2half_rn(v);
}

// Four neighbouring columns, the first `left` of them.
__device__ __forceinline__ void store_c4(const NarrowParams& p, int64_t at, int left,
                                         const float (&v)[4]) {
  if (p.vec_c && left >= 4) {
    if (p.c_dtype == MHR_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.C) + at) =
          make_float4(v[0], v[1], v[2], v[3]);
      return;
    }
    uint32_t w[2];
    if (p.c_dtype == MHR_BF16) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]);
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2], v[3]);
      w[0] = *reinterpret_cast<const uint32_t*>(&a);
      w[1] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
      w[0] = *reinterpret_cast<const uint32_t*>(&a);
      w[1] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.C) + at) = make_uint2(w[0], w[1]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) store_c(p, at + i, v[i]);
}

// 8 values of a row from column k on; zeros past the end.  (No read-only loads: the
// kernel before, which may write them, still runs when this one starts.)
template <typename T>
__device__ __forceinline__ void load_row8(const T* row, int k, int K, bool vec, float (&v)[8]) {
  if (vec && k + 8 <= K) {
    alignas(16) T t[8];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(t) / 16); ++i)
      reinterpret_cast<uint4*>(t)[i] = reinterpret_cast<const uint4*>(row + k)[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_float(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k + i < K ? to_float(row[k + i]) : 0.f;
  }
}

// Rows of a plain A into `staged`, as gemm_mxfp4_quantize would pack them and TMA
// and the scales' copies would bring them: per stage of 256 columns a scale tile
// pair (1 KB), and for all stages behind them 128 bytes a row, swizzled.  A warp
// takes a stage of a row, 8 columns a lane.
template <typename T>
__device__ __forceinline__ void quantize_part(const NarrowParams& p, uint8_t* staged, int m0,
                                              int kb0, int kb1, int warp, int warps, int lane) {
  const int kn = kb1 - kb0, rows = min(p.nt, p.M - m0);
  uint8_t* codes = staged + kn * SF_BYTES;
  for (int t = warp; t < rows * kn; t += warps) {
    const int m = t / kn, s = t - m * kn;
    const T* row = static_cast<const T*>(p.a) + (m0 + m) * p.lda;
    float v[8];
    load_row8<T>(row, (kb0 + s) * 256 + lane * 8, p.K, p.vec_a != 0, v);
    uint32_t amax = __float_as_uint(max_abs8(v));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t code = scale_code(amax);
    const int block = lane >> 2;
    *reinterpret_cast<uint32_t*>(codes + (s * p.nt + m) * 128 + ((block ^ (m & 7)) << 4) +
                                 (lane & 3) * 4) =
        code == 255u ? 0u : encode8(v, scale_inverse(code));
    if ((lane & 3) == 0)
      staged[s * SF_BYTES + (block >> 2) * 512 + (m & 31) * 16 + (m >> 5) * 4 + (block & 3)] =
          static_cast<uint8_t>(code);
  }
}

// Warp roles: 0 TMA producer, 1 TMEM allocator and MMA issuer, 2-5 epilogue
// (TMEM lanes 32 * (warp % 4) on); with a plain A (type T), 2-15 quantise it
// first.  Every wait is bounded; a role that gives up records it in the status
// word and raises the CTA's abort flag.
template <typename T>
__global__ void __launch_bounds__(std::is_void<T>::value ? THREADS : PLAIN_THREADS, 2)
    mxfp4_narrow_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB, const NarrowParams p) {
  constexpr bool PLAIN = !std::is_void<T>::value;
  extern __shared__ uint8_t smem_raw[];
  __shared__ alignas(8) uint64_t bars[2 * MAX_STAGES + 2];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t abase = smem_u32(smem), sbase = abase + (PLAIN ? p.a_bytes : 0);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (MAX_STAGES + s); };
  const uint32_t acc_bar = bar0 + 8u * (2 * MAX_STAGES);
  const uint32_t a_bar = bar0 + 8u * (2 * MAX_STAGES + 1);  // plain A: quantised
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / p.split;
  const int tile_m = tile / p.tiles_n;
  const int n0 = (tile - tile_m * p.tiles_n) * W_ROWS, m0 = tile_m * p.nt;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.num_kb) * rank / p.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.num_kb) * (rank + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(acc_bar, 1);
    mbar_init(a_bar, PLAIN_THREADS / 32 - 2);
    abort_flag = 0;
    fence_mbar_init();
    if (!PLAIN) tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
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
  grid_launch_dependents();  // (they wait for this grid's end before they read or write)
  auto give_up = [&](uint32_t bit) {  // by one thread
    if (!abort_flag) atomicOr(p.status, bit);
    abort_flag = 1;
  };
  const int x_bytes = PLAIN ? 0 : p.nt * BK_BYTES;  // of A in a ring stage
  const uint32_t off_x = W_BYTES, off_sfb = W_BYTES + x_bytes, off_sfa = off_sfb + SF_BYTES;
  auto sf_bytes = [&](int kb) { return static_cast<uint32_t>(min(2, p.kt - 2 * kb)) * 512u; };

  if (warp == 0) {
    auto load_b = [&](uint32_t st, uint32_t bar, int kb) {
      tma_load_2d(st, &tmB, bar, kb * BK_BYTES, n0);
      bulk_load(st + off_sfb, p.sfb + (static_cast<int64_t>(n0 / 128) * p.kt + 2 * kb) * 512,
                sf_bytes(kb), bar);
    };
    auto load_a = [&](uint32_t st, uint32_t bar, int kb) {
      if (PLAIN) return;
      tma_load_2d(st + off_x, &tmA, bar, kb * BK_BYTES, m0);
      bulk_load(st + off_sfa, p.sfa + (static_cast<int64_t>(m0 / 128) * p.kt + 2 * kb) * 512,
                sf_bytes(kb), bar);
    };
    auto tx = [&](int kb) { return W_BYTES + x_bytes + (PLAIN ? 1u : 2u) * sf_bytes(kb); };
    const bool stall = p.inject_stall && blockIdx.x == 0;  // test hook: stage 0 never fills
    // The first stages' B before the kernel before this one (A's quantisation)
    // has finished, where that is known not to write B.
    const int ahead = min(p.stages, kb1 - kb0);
    if (!p.early_b) grid_dependency_wait();
    if (elect_one()) {
      for (int i = 0; i < ahead; ++i) {
        mbar_arrive_expect_tx(full_bar(i), tx(kb0 + i));
        if (!(stall && i == 0)) load_b(sbase + i * p.stage_bytes, full_bar(i), kb0 + i);
      }
    }
    __syncwarp();
    if (p.early_b) grid_dependency_wait();
    if (elect_one()) {
      for (int i = stall ? 1 : 0; i < ahead; ++i)
        load_a(sbase + i * p.stage_bytes, full_bar(i), kb0 + i);
    }
    __syncwarp();
    int it = ahead;
    uint32_t s = 0, ph = 0;  // of the stage to fill again: its first MMAs done
    for (; kb0 + it < kb1; ++it) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(empty_bar(s), ph, limit, &abort_flag))) {
        if (lane == 0) give_up(kErrTimeoutProducer);
        break;
      }
      if (elect_one()) {
        mbar_arrive_expect_tx(full_bar(s), tx(kb0 + it));
        load_b(sbase + s * p.stage_bytes, full_bar(s), kb0 + it);
        load_a(sbase + s * p.stage_bytes, full_bar(s), kb0 + it);
      }
      __syncwarp();
      if (++s == static_cast<uint32_t>(p.stages)) {
        s = 0;
        ph ^= 1u;
      }
    }
    if (lane == 0) {
      // This CTA's copies in flight have landed before it goes on to leave.
      volatile int never = 0;
      for (int i = max(0, it - p.stages); i < it; ++i) {
        if (stall && i == 0) {  // counted as done once the MMA issuer has given up on it
          mbar_wait_bounded(full_bar(0), 0, 2 * limit, &abort_flag);
          mbar_complete_tx(full_bar(0), tx(kb0));
        }
        if (!mbar_wait_bounded(full_bar(i % p.stages), (i / p.stages) & 1u, limit, &never))
          atomicOr(p.status, kErrTimeoutDrain);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t id0 = make_idesc_mxf4(W_ROWS, p.nt, 0), id2 = make_idesc_mxf4(W_ROWS, p.nt, 2);
    uint32_t s = 0, ph = 0;  // ring position
    bool ready = true;
    if (PLAIN) ready = mbar_wait_bounded(a_bar, 0, limit, &abort_flag);
    for (int it = 0; kb0 + it < kb1; ++it) {
      // (a stage's scales have TMEM columns of their own: whoever read them
      // last had finished before the producer filled the stage again)
      const bool ok = ready && mbar_wait_bounded(full_bar(s), ph, limit, &abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) give_up(kErrTimeoutMma);
        break;
      }
      tc_fence_after();
      const int kb = kb0 + it;
      const uint32_t w = desc_lo(sbase + s * p.stage_bytes), cb = w + (off_sfb >> 4);
      const uint32_t part = desc_lo(abase);
      const uint32_t x = PLAIN ? part + (((kb1 - kb0) * SF_BYTES + it * p.nt * BK_BYTES) >> 4)
                               : w + (off_x >> 4);
      const uint32_t ca = PLAIN ? part + ((it * SF_BYTES) >> 4) : w + (off_sfa >> 4);
      const uint32_t sfb = tmem + p.sf_col + s * 16, sfa = sfb + 8;
      const int left = p.blocks - kb * 8;
      const uint32_t first = it > 0 ? 1u : 0u;
      if (elect_one()) {
        if (left >= 8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            copy_scale_tile<1>(sfb + 4 * i, cb + 32 * i);
            copy_scale_tile<1>(sfa + 4 * i, ca + 32 * i);
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_mxf4<1>(tmem, w + 2 * kk, x + 2 * kk, kk & 1 ? id2 : id0, sfb + 4 * (kk >> 1),
                        sfa + 4 * (kk >> 1), kk > 0 ? 1u : first);
        } else {  // the last stage of K
          const int tiles = left > 4 ? 2 : 1, mmas = (left + 1) / 2;
          for (int i = 0; i < tiles; ++i) {
            copy_scale_tile<1>(sfb + 4 * i, cb + 32 * i);
            copy_scale_tile<1>(sfa + 4 * i, ca + 32 * i);
          }
          for (int kk = 0; kk < mmas; ++kk)
            mma_mxf4<1>(tmem, w + 2 * kk, x + 2 * kk, kk & 1 ? id2 : id0, sfb + 4 * (kk >> 1),
                        sfa + 4 * (kk >> 1), kk > 0 ? 1u : first);
        }
        mma_commit(empty_bar(s));
      }
      __syncwarp();
      if (++s == static_cast<uint32_t>(p.stages)) {
        s = 0;
        ph ^= 1u;
      }
    }
    if (elect_one()) mma_commit(acc_bar);
    __syncwarp();
    volatile int never = 0;
    if (!mbar_wait_bounded(acc_bar, 0, limit, &never) && lane == 0)
      atomicOr(p.status, kErrTimeoutDrain);
  } else {
    const int q = warp & 3;
    grid_dependency_wait();  // C may be read or written by the kernel before this one
    if constexpr (PLAIN) {
      quantize_part<T>(p, smem, m0, kb0, kb1, warp - 2, PLAIN_THREADS / 32 - 2, lane);
      fence_proxy_async_smem();  // for the MMAs and scale copies that read it
      __syncwarp();
      if (lane == 0) mbar_arrive(a_bar);
    }
    if (warp < 6) {
      const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(acc_bar, 0, limit, &abort_flag));
      if (!ok && lane == 0) give_up(kErrTimeoutEpilogue);
      __syncwarp();
      tc_fence_after();
      const int n = n0 + q * 32 + lane;
      const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16);
      // [row of A][128]: the ring is idle by now
      float* red = reinterpret_cast<float*>(smem + (PLAIN ? p.a_bytes : 0));
      if (ok && kb0 < kb1) {
        for (int j0 = 0; j0 < p.nt; j0 += 8) {
          uint32_t r[8];
          tmem_ld_8cols(taddr + j0, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (p.split > 1)
              red[(j0 + j) * W_ROWS + q * 32 + lane] = __uint_as_float(r[j]);
            else if (m0 + j0 + j < p.M && n < p.N)
              store_c(p, static_cast<int64_t>(m0 + j0 + j) * p.ldc + n, __uint_as_float(r[j]));
          }
        }
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (p.split > 1) {
    cluster_sync_all();
    if (!abort_flag && warp >= 2 && warp < 6) {
      // Partial sums of the cluster, added in rank order: 4 columns a thread.
      const int quads = min(p.nt, p.M - m0) * (W_ROWS / 4);
      for (int g = rank * 128 + threadIdx.x - 64; g < quads; g += p.split * 128) {
        const uint32_t addr = sbase + g * 16;
        float4 part[MAX_SPLIT];  // (all reads on their way before the first is added)
#pragma unroll
        for (int r = 0; r < MAX_SPLIT; ++r)
          if (r < p.split)
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(part[r].x), "=f"(part[r].y), "=f"(part[r].z), "=f"(part[r].w)
                         : "r"(mapa_shared(addr, r))
                         : "memory");
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < MAX_SPLIT; ++r)
          if (r < p.split) {
            sum[0] += part[r].x;
            sum[1] += part[r].y;
            sum[2] += part[r].z;
            sum[3] += part[r].w;
          }
        const int m = m0 + g / (W_ROWS / 4), n = n0 + g % (W_ROWS / 4) * 4;
        store_c4(p, static_cast<int64_t>(m) * p.ldc + n, p.N - n, sum);
      }
    }
    cluster_sync_all();  // no CTA leaves while another reads its partial sums
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

}  // namespace

namespace {

// (static state: by device, under the library's lock)
// CTAs that run at once in clusters of `split`, one an SM.  (Clusters pack into an
// SM group or leave some of its SMs out, so it is less than the SMs: of 128 CTAs
// in clusters of 8, eight wait.)
template <typename T>
cudaError_t allow_smem(int device) {
  static bool done[64];
  if (device < 64 && done[device]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(
      mxfp4_narrow_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT - 1024);
  if (e == cudaSuccess && device < 64) done[device] = true;
  return e;
}
template <typename T>
cudaError_t slots_t(int device, int split, int* slots) {
  constexpr bool PLAIN = !std::is_void<T>::value;
  auto kern = mxfp4_narrow_kernel<T>;
  static int known[64][MAX_SPLIT + 1];
  int* at = device < 64 ? &known[device][split] : nullptr;
  if (!at || !*at) {
    cudaError_t e = allow_smem<T>(device);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split * 256);
    cfg.blockDim = dim3(PLAIN ? PLAIN_THREADS : THREADS);
    cfg.dynamicSmemBytes = SMEM_LIMIT - 1024;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg)) != cudaSuccess) return e;
    *slots = clusters * split;
    if (at) *at = *slots;
  } else {
    *slots = *at;
  }
  return cudaSuccess;
}

cudaError_t slots_of(bool plain, int a_dtype, int device, int split, int* slots) {
  if (!plain) return slots_t<void>(device, split, slots);
  switch (a_dtype) {
    case MHR_F32: return slots_t<float>(device, split, slots);
    case MHR_BF16: return slots_t<__nv_bfloat16>(device, split, slots);
    default: return slots_t<__half>(device, split, slots);
  }
}

template <typename T>
cudaError_t launch_t(const CUtensorMap& tmA, const CUtensorMap& tmB, const NarrowParams& p,
                     int64_t tiles, int smem, int device, cudaStream_t s) {
  constexpr bool PLAIN = !std::is_void<T>::value;
  auto kern = mxfp4_narrow_kernel<T>;
  if (const cudaError_t e = allow_smem<T>(device); e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.split));
  cfg.blockDim = dim3(PLAIN ? PLAIN_THREADS : THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  note_main_kernel(PLAIN ? "mxfp4_narrow_kernel<plain>" : "mxfp4_narrow_kernel",
                   static_cast<int>(tiles * p.split), static_cast<int>(tiles));
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tmA, tmB, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Tiles and K parts of a product; the part of A that a CTA quantises if it does.
// As many parts as can run at once: GB300, 1 x 4096 x 4096 in 1 / 2 / 4 / 6 parts
// 7.0 / 6.5 / 6.0 / 5.6 us, 24 x 11008 x 4096 in 1 / 2 / 3 8.6 / 8.9 / 8.8 us; in 4,
// which do not all run at once, it took half as long again as in 3.
cudaError_t plan_narrow(int64_t M, int64_t N, int64_t K, bool plain, int a_dtype, int device,
                        NarrowParams* p, int64_t* tiles) {
  p->M = static_cast<int32_t>(M);
  p->N = static_cast<int32_t>(N);
  p->K = static_cast<int32_t>(K);
  p->nt = M >= MAX_NT ? MAX_NT : static_cast<int32_t>((M + 7) / 8 * 8);
  p->tiles_n = static_cast<int32_t>((N + W_ROWS - 1) / W_ROWS);
  p->blocks = static_cast<int32_t>(blocks_of(K));
  p->kt = static_cast<int32_t>(scale_tiles(K));
  p->num_kb = (p->kt + 1) / 2;
  *tiles = (M + p->nt - 1) / p->nt * p->tiles_n;
  for (p->split = p->num_kb < MAX_SPLIT ? p->num_kb : MAX_SPLIT; p->split > 1; --p->split) {
    int slots = 0;
    const cudaError_t e = slots_of(plain, a_dtype, device, p->split, &slots);
    if (e != cudaSuccess) return e;
    if (*tiles * p->split <= (p->nt <= PAIR_NT ? 2 : 1) * slots) break;
  }
  p->a_bytes = (p->num_kb + p->split - 1) / p->split * (SF_BYTES + p->nt * BK_BYTES);
  return cudaSuccess;
}

}  // namespace

cudaError_t narrow_quantizes(int64_t M, int64_t N, int64_t K, int a_dtype, int device, bool* yes) {
  *yes = false;
  if (M > PLAIN_ROWS) return cudaSuccess;
  NarrowParams p;
  int64_t tiles;
  const cudaError_t e = plan_narrow(M, N, K, true, a_dtype, device, &p, &tiles);
  *yes = p.a_bytes <= PLAIN_BYTES && M * ((p.num_kb + p.split - 1) / p.split) <= PLAIN_TASKS;
  return e;
}

cudaError_t narrow_time(int64_t M, int64_t N, int64_t K, int sms, int device, double* us) {
  NarrowParams p;
  int64_t tiles;
  const cudaError_t e = plan_narrow(M, N, K, false, 0, device, &p, &tiles);
  if (e != cudaSuccess) return e;
  const int64_t rounds = (tiles * p.split + sms - 1) / sms;
  const int stages = (p.num_kb + p.split - 1) / p.split;
  *us = 4.9 + 0.018 * p.nt + static_cast<double>(rounds) * stages * (0.2 + 0.0009 * p.nt);
  return cudaSuccess;
}

cudaError_t launch_narrow(const ProductArgs& a, const DeviceCtl& ctl, cudaStream_t s) {
  NarrowParams p;
  int64_t tiles;
  const bool plain = a.a_plain != nullptr;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = plan_narrow(a.M, a.N, a.K, plain, a.a_dtype, device, &p, &tiles);
  if (e != cudaSuccess) return e;
  if (tiles * p.split > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int room = (p.nt <= PAIR_NT ? SMEM_LIMIT / 2 : SMEM_LIMIT) - 1024 - 1024 -
                   (plain ? p.a_bytes : 0);
  p.stage_bytes = W_BYTES + (plain ? SF_BYTES : p.nt * BK_BYTES + 2 * SF_BYTES);
  p.stages = room / p.stage_bytes;
  p.sf_col = (p.nt + 31) / 32 * 32;
  const int sets = static_cast<int>(TMEM_COLS - p.sf_col) / 16;
  if (p.stages > sets) p.stages = sets;
  if (p.stages > MAX_STAGES) p.stages = MAX_STAGES;
  p.early_b = a.after_quantize;
  p.sfa = a.sfa;
  p.sfb = a.sfb;
  p.a = a.a_plain;
  p.lda = a.lda;
  const int64_t size = a.a_dtype == MHR_F32 ? 4 : 2;
  p.vec_a = reinterpret_cast<uintptr_t>(a.a_plain) % 16 == 0 && a.lda * size % 16 == 0;
  p.C = a.C;
  p.ldc = a.ldc;
  p.c_dtype = a.c_dtype;
  const int64_t c_size = a.c_dtype == MHR_F32 ? 4 : 2;
  p.vec_c = reinterpret_cast<uintptr_t>(a.C) % (4 * c_size) == 0 && a.ldc % 4 == 0;
  p.status = ctl.status;
  p.wait_limit_ns = ctl.wait_limit_ns;
  p.inject_stall = ctl.inject_stall;
  const int64_t row_bytes = static_cast<int64_t>(p.blocks) * 16;
  CUtensorMap tmA, tmB;
  if (encode_tmap_2d(&tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.B, row_bytes, a.N, a.ldb, BK_BYTES,
                     W_ROWS, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  tmA = tmB;
  if (!plain && encode_tmap_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.A, row_bytes, a.M, a.lda,
                               BK_BYTES, p.nt, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const int smem = p.stages * p.stage_bytes + (plain ? p.a_bytes : 0) + 1024;
  if (!plain) return launch_t<void>(tmA, tmB, p, tiles, smem, device, s);
  switch (a.a_dtype) {
    case MHR_F32: return launch_t<float>(tmA, tmB, p, tiles, smem, device, s);
    case MHR_BF16: return launch_t<__nv_bfloat16>(tmA, tmB, p, tiles, smem, device, s);
    default: return launch_t<__half>(tmA, tmB, p, tiles, smem, device, s);
  }
}

}  // namespace mx
}  // namespace mhr
