// The stable order of (token, slot) pairs by expert, and where each expert's part
// starts (gemm_routed_sort): a counting sort in one launch.
//
// The warps of one cluster take contiguous runs of entries.  Each counts its run's
// experts in a row of counters of its own, so nothing depends on the order of
// atomics; the counters' sums over warps, CTAs (through distributed shared memory)
// and experts give every warp its first place in each expert's part; a second walk
// puts the positions there, equal experts of 32 entries in their order.
// Bound by latency: a run's loads, 16 a lane, go out together, and a bin's 32
// counters, and 8 or 16 CTAs' totals, are read at once.  GB300: 131072 entries of 256
// experts in 11.8 us (36 with one load and one counter at a time and 8 CTAs), 64 in 5.
#include <cuda_runtime.h>

#include <cstdint>

#include "mhr_device.cuh"
#include "routed_internal.h"

namespace mhr {
namespace routed {
namespace {

constexpr uint32_t ALL = 0xffffffffu;
constexpr int MAX_CTAS = 16;  // (above 8: not every GPU's clusters)
constexpr int MAX_WARPS = 32;
constexpr int EACH = 16;      // entries a lane loads at once

__device__ __forceinline__ uint32_t ld_shared_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Shared memory: counters (warps x bins), and this CTA's total of each bin.
template <int CTAS>
__global__ void __launch_bounds__(MAX_WARPS * 32, 1)
    sort_kernel(const int32_t* experts, int64_t n, int E, int32_t* offsets, int32_t* order) {
  extern __shared__ uint32_t counters[];
  const int bins = E + 1;  // the last: outside 0 .. E-1
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x;  // the grid is one cluster
  uint32_t* mine = counters + warp * bins;
  uint32_t* total = counters + warps * bins;
  __shared__ uint32_t warp_sums[MAX_WARPS];

  for (int i = threadIdx.x; i < warps * bins; i += blockDim.x) counters[i] = 0;
  __syncthreads();
  grid_dependency_wait();

  const int64_t run = (n + 32 * warps * CTAS - 1) / (32 * warps * CTAS) * 32;
  const int64_t from = min(n, (static_cast<int64_t>(rank) * warps + warp) * run);
  const int64_t to = min(n, from + run);
  // f(this lane's entry's bin, its position, whether there is one), 32 entries at a time
  auto walk = [&](const auto& f) {
    for (int64_t i0 = from; i0 < to; i0 += 32 * EACH) {
      int e[EACH];
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        const int64_t i = i0 + 32 * j + lane;
        e[j] = i < to ? experts[i] : -1;
      }
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        const int64_t i = i0 + 32 * j;
        if (i < to) f(e[j] >= 0 && e[j] < E ? e[j] : E, i + lane, i + lane < to);
      }
    }
  };
  walk([&](int e, int64_t, bool in) {
    if (in) atomicAdd(&mine[e], 1u);
  });
  __syncthreads();
  // f(warp w's counter of bin b), in order
  auto counters_of = [&](int b, const auto& f) {
    for (int w0 = 0; w0 < warps; w0 += 8) {
      uint32_t c[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) c[w] = counters[(w0 + w) * bins + b];
#pragma unroll
      for (int w = 0; w < 8; ++w) f(c[w], w0 + w);
    }
  };
  for (int b = threadIdx.x; b < bins; b += blockDim.x) {
    uint32_t sum = 0;
    counters_of(b, [&](uint32_t c, int) { sum += c; });
    total[b] = sum;
  }
  if constexpr (CTAS > 1)
    cluster_sync_all();
  else
    __syncthreads();
  // Over the CTAs and the bins: runs of blockDim.x bins, with a running base.  Each
  // counter becomes its warp's first place.
  uint32_t base = 0;
  for (int b0 = 0; b0 < bins; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    uint32_t all = 0, before = 0;
    if (b < bins) {
      if constexpr (CTAS > 1) {
        const uint32_t at = smem_u32(total + b);
        uint32_t c[CTAS];
#pragma unroll
        for (int r = 0; r < CTAS; ++r) c[r] = ld_shared_cluster(mapa_shared(at, r));
#pragma unroll
        for (int r = 0; r < CTAS; ++r) {
          before += r < rank ? c[r] : 0;
          all += c[r];
        }
      } else {
        all = total[b];
      }
    }
    uint32_t scan = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(ALL, scan, d);
      if (lane >= d) scan += o;
    }
    if (lane == 31) warp_sums[warp] = scan;
    __syncthreads();
    uint32_t sums = lane < warps ? warp_sums[lane] : 0;  // of the warps, by every warp
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(ALL, sums, d);
      if (lane >= d) sums += o;
    }
    const uint32_t lower = warp ? __shfl_sync(ALL, sums, (warp - 1) & 31) : 0;
    const uint32_t block = __shfl_sync(ALL, sums, 31);
    if (b < bins) {
      const uint32_t first = base + lower + scan - all;
      if (rank == 0) offsets[b] = static_cast<int32_t>(first);  // (bin E starts at offsets[E])
      uint32_t place = first + before;
      counters_of(b, [&](uint32_t c, int w) {
        counters[w * bins + b] = place;
        place += c;
      });
    }
    base += block;
    __syncthreads();
  }
  if constexpr (CTAS > 1)  // this CTA has read the others' totals
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const int bits = 32 - __clz(E);
  walk([&](int e, int64_t i, bool in) {
    // Lanes of the same bin, bit by bit: a warp's match takes the SM some 70 cycles, a vote
    // one or two.
    uint32_t same = __ballot_sync(ALL, in);
    for (int k = 0; k < bits; ++k) {
      const bool set = e >> k & 1;
      const uint32_t vote = __ballot_sync(ALL, set);
      same &= set ? vote : ~vote;
    }
    uint32_t at = 0;
    if (in) at = mine[e];
    __syncwarp();
    if (in) {
      if (__ffs(same) - 1 == lane) mine[e] = at + __popc(same);
      at += __popc(same & ((1u << lane) - 1));
      // (past n only where another kernel writes the entries meanwhile)
      if (at < n) order[at] = static_cast<int32_t>(i);
    }
    __syncwarp();
  });
  // No CTA leaves while another may still read its totals.
  if constexpr (CTAS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int CTAS>
cudaError_t launch_ctas(const int32_t* experts, int64_t n, int64_t E, int32_t* offsets,
                        int32_t* order, int warps, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CTAS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CTAS);
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
  cfg.dynamicSmemBytes = (static_cast<size_t>(warps) + 1) * (E + 1) * sizeof(uint32_t);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = CTAS > 1 ? 2 : 1;
  constexpr size_t most = (MAX_WARPS + 1) * (MAX_PARTS + 1) * sizeof(uint32_t);  // 132 KB
  auto kern = sort_kernel<CTAS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(most));
  if (e == cudaSuccess && CTAS > 8)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  note_launch();
  e = cudaLaunchKernelEx(&cfg, kern, experts, n, static_cast<int>(E), offsets, order);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_sort(const int32_t* experts, int64_t n, int64_t E, int32_t* offsets,
                        int32_t* order, cudaStream_t s) {
  // GB300, one CTA against a cluster of 16: 4096 entries of 256 experts 7.9 / 7.3 us,
  // 16384 15.8 / 7.4.  Warps by what is left to each: their counters are summed up twice.
  const int64_t chunks = (n + 31) / 32;
  if (chunks > 64) {
    int warps = 8;
    while (warps < MAX_WARPS && warps * MAX_CTAS * 4 < chunks) warps *= 2;
    return launch_ctas<MAX_CTAS>(experts, n, E, offsets, order, warps, s);
  }
  int warps = 8;
  while (warps < MAX_WARPS && warps < chunks) warps *= 2;
  return launch_ctas<1>(experts, n, E, offsets, order, warps, s);
}

}  // namespace routed
}  // namespace mhr
