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
// v stays in 32 bits on the way: for the tensor cores it is written as a sum of 16-bit
// terms (hi + lo, and a third for fp32 results of bf16).
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
      for (int n = n0 + threadIdx.x; n < n1; n += ROW_THREADS) out[n] = y[n];
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
    // lane 8 g' + c sends row g' of the group to CTA c
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

}  // namespace

int64_t adapters_scratch(const AdapterArgs&) { return 0; }

cudaError_t launch_adapters(const AdapterArgs& a, void*, const DeviceCtl&, cudaStream_t s) {
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
  return a.dtype == MHR_BF16 ? launch_out<__nv_bfloat16>(a, p, s) : launch_out<__half>(a, p, s);
}

}  // namespace routed
}  // namespace mhr
