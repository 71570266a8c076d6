// The stable order of (token, slot) pairs by expert, and where each expert's part
// starts (gemm_routed_sort): a counting sort in one launch.
//
// The warps of one cluster take contiguous runs of entries.  Each counts its run's
// experts in a row of counters of its own, so nothing depends on the order of
// atomics; the counters' sums over warps, CTAs (through distributed shared memory)
// and experts give every warp its first place in each expert's part; a second walk
// puts the positions there, equal experts of 32 entries by match and popcount.
#include <cuda_runtime.h>

#include <cstdint>

#include "mhr_device.cuh"
#include "routed_internal.h"

namespace mhr {
namespace routed {
namespace {

constexpr uint32_t ALL = 0xffffffffu;
constexpr int MAX_CTAS = 8;
constexpr int MAX_WARPS = 32;

__device__ __forceinline__ uint32_t ld_shared_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Shared memory: counters (warps x bins), this CTA's total of each bin (bins), and
// the bins' starts (bins).
__global__ void __launch_bounds__(MAX_WARPS * 32, 1)
    sort_kernel(const int32_t* experts, int64_t n, int E, int32_t* offsets, int32_t* order) {
  extern __shared__ uint32_t counters[];
  const int bins = E + 1;  // the last: outside 0 .. E-1
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ctas = gridDim.x, rank = blockIdx.x;  // the grid is one cluster
  uint32_t* mine = counters + warp * bins;
  uint32_t* total = counters + warps * bins;
  uint32_t* start = total + bins;
  __shared__ uint32_t warp_sums[MAX_WARPS];

  for (int i = threadIdx.x; i < warps * bins; i += blockDim.x) counters[i] = 0;
  __syncthreads();
  grid_dependency_wait();

  const int64_t run = (n + 32 * warps * ctas - 1) / (32 * warps * ctas) * 32;
  const int64_t from = min(n, (static_cast<int64_t>(rank) * warps + warp) * run);
  const int64_t to = min(n, from + run);
  auto bin_at = [&](int64_t i) {
    const int e = i < to ? experts[i] : -1;
    return e >= 0 && e < E ? e : E;
  };
  for (int64_t i = from; i < to; i += 32) {
    const bool in = i + lane < to;
    const int e = bin_at(i + lane);
    const uint32_t same = __match_any_sync(ALL, in ? e : -1);
    if (in && __ffs(same) - 1 == lane) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // Over the warps: each counter becomes the entries of the warps before it.
  for (int b = threadIdx.x; b < bins; b += blockDim.x) {
    uint32_t sum = 0;
    for (int w = 0; w < warps; ++w) {
      const uint32_t c = counters[w * bins + b];
      counters[w * bins + b] = sum;
      sum += c;
    }
    total[b] = sum;
  }
  if (ctas > 1)
    cluster_sync_all();
  else
    __syncthreads();
  // Over the CTAs and the bins: runs of blockDim.x bins, with a running base.
  uint32_t base = 0;
  for (int b0 = 0; b0 < bins; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    uint32_t all = 0, before = 0;
    if (b < bins) {
      if (ctas > 1) {
        const uint32_t at = smem_u32(total + b);
        for (int r = 0; r < ctas; ++r) {
          const uint32_t c = ld_shared_cluster(mapa_shared(at, r));
          if (r < rank) before += c;
          all += c;
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
    uint32_t lower = 0, block = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) lower += warp_sums[w];
      block += warp_sums[w];
    }
    if (b < bins) {
      const uint32_t first = base + lower + scan - all;
      start[b] = first + before;
      if (rank == 0) offsets[b] = static_cast<int32_t>(first);  // (bin E starts at offsets[E])
    }
    base += block;
    __syncthreads();
  }
  // No CTA leaves while another may still read its totals.
  if (ctas > 1) cluster_sync_all();
  for (int64_t i = from; i < to; i += 32) {
    const bool in = i + lane < to;
    const int e = bin_at(i + lane);
    const uint32_t same = __match_any_sync(ALL, in ? e : -1);
    uint32_t at = 0;
    if (in) at = start[e] + mine[e] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (in) {
      // (past n only where another kernel writes the entries meanwhile)
      if (at < n) order[at] = static_cast<int32_t>(i + lane);
      if (__ffs(same) - 1 == lane) mine[e] += __popc(same);
    }
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_sort(const int32_t* experts, int64_t n, int64_t E, int32_t* offsets,
                        int32_t* order, cudaStream_t s) {
  const int64_t chunks = (n + 31) / 32;
  int warps = 8;
  while (warps < MAX_WARPS && warps < chunks) warps *= 2;
  const int ctas = chunks > 4 * MAX_WARPS ? MAX_CTAS : 1;
  const size_t bins = static_cast<size_t>(E) + 1;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
  cfg.dynamicSmemBytes = (warps + 2) * bins * sizeof(uint32_t);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  constexpr size_t most = (MAX_WARPS + 2) * (MAX_PARTS + 1) * sizeof(uint32_t);  // 136 KB
  cudaError_t e = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(most));
  if (e != cudaSuccess) return e;
  note_launch();
  e = cudaLaunchKernelEx(&cfg, sort_kernel, experts, n, static_cast<int>(E), offsets, order);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace routed
}  // namespace mhr
