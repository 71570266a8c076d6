// Quantisation to microscaled 4-bit floats (the format is in mxfp4_common.cuh):
// per block of 32 values the scale s = 2^(floor(log2 max|x|) - 2), then each
// code is x / s rounded to e2m1.  s is a power of two, so x / s = x * 2^-k is
// exact and the only rounding is the last one.
//
// Bound by HBM: X is read once, 17/32 byte a value written (plus `values`,
// X's size again, when asked for).
#include "mhr_gemm.h"
#include "mhr_mxfp4.h"
#include "mxfp4_common.cuh"

namespace mhr {
namespace mx {
namespace {

// Launched as a programmatic dependent: the kernel before has to finish before
// anything is read or written here, and only then may the kernel after this one
// start -- whatever came before this kernel is complete by then, as the narrow
// product's early loads of B need (ProductArgs::after_quantize).
__device__ __forceinline__ void start_in_order() {
  grid_dependency_wait();
  grid_launch_dependents();
}

// The values that 8 codes stand for: e2m1 is exact in f16, and f16 -> fp32 and
// the product with a power of two are exact too.
__device__ __forceinline__ void decode8(uint32_t w, float scale, float (&v)[8]) {
  const uint32_t h[4] = {e2m1_to_f16x2<0>(w), e2m1_to_f16x2<1>(w), e2m1_to_f16x2<2>(w),
                         e2m1_to_f16x2<3>(w)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x * scale;
    v[2 * i + 1] = f.y * scale;
  }
}

// 8 values of type T as loaded, and as floats.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
      w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  }
  // one value at a time, zeros from `left` on
  __device__ __forceinline__ void load(const T* p, int64_t left) {
    alignas(16) T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = i < left ? p[i] : from_float<T>(0.f);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
      w[i] = reinterpret_cast<const uint4*>(t)[i];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_float(reinterpret_cast<const T*>(w)[i]);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    alignas(16) T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = from_float<T>(v[i]);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
      w[i] = reinterpret_cast<const uint4*>(t)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
  }
  __device__ __forceinline__ void store(T* p, int64_t left) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = reinterpret_cast<const T*>(w)[i];
  }
};

struct RowParams {
  const void* x;
  int64_t ldx, rows, cols;
  uint8_t* data;
  int64_t ldd;
  uint8_t* scales;
  void* values;
  int64_t ldv;
  int64_t kt;       // scale tiles along a row
  uint32_t chunks;  // of 256 columns along a row
};

constexpr int ROW_CHUNK = 256;  // columns of a warp: 8 a lane
constexpr int ROW_STEPS = 4;    // rows of a warp

// Blocks along the rows: one pass, bound by HBM.  A warp takes 256 columns (16 bytes a lane of a 16-bit
// type) of the four rows r, r + 32, r + 64 and r + 96 of a tile of 128: their
// scales are neighbours in the tile and go out 16 bytes at a time.  All loads
// first; a block is four neighbouring lanes, its maximum two shuffles.  Rows past
// the last up to a multiple of 128 get zero scales (the tiles are written whole).
// GB300, call after call: 8192 x 8192 bf16 25.9 us (6.6 TB/s), with values 46.8 (6.5
// TB/s); fp32 37.9 (8.0 TB/s, some of it the last call's input still in L2); 333 x
// 4104 bf16 2.3 us and one row of 4096 2.2, a launch's time.
template <typename T, bool VEC, bool VALUES>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const RowParams p) {
  start_in_order();
  const int lane = threadIdx.x & 31;
  // (32-bit division: fewer than 2^31 warps of a launch, see launch_t)
  const uint32_t task = blockIdx.x * 8u + (threadIdx.x >> 5), set = task / p.chunks;
  const int64_t row0 = static_cast<int64_t>(set >> 5) * 128 + (set & 31);
  if (row0 >= (p.rows + 127) / 128 * 128) return;
  const int64_t c = static_cast<int64_t>(task - set * p.chunks) * ROW_CHUNK + lane * 8;
  const T* x = static_cast<const T*>(p.x) + c;
  uint8_t* data = p.data + row0 * p.ldd + c / 2;
  uint32_t codes4 = 0;  // the scales' codes of the rows' blocks, a byte a row
  // Whole rows take their loads in one go, with no branch and no conversion
  // between them (either makes each wait for the one before).
  const bool whole = VEC && row0 + 96 < p.rows && c - lane * 8 + ROW_CHUNK <= p.cols;
  Raw8<T> raw[ROW_STEPS];
  if (whole) {
#pragma unroll
    for (int i = 0; i < ROW_STEPS; ++i) raw[i].load(x + (row0 + 32 * i) * p.ldx);
  } else {
#pragma unroll
    for (int i = 0; i < ROW_STEPS; ++i) {
      const int64_t row = row0 + 32 * i, left = row < p.rows ? p.cols - c : 0;
      if (VEC && left >= 8)
        raw[i].load(x + row * p.ldx);
      else
        raw[i].load(x + row * p.ldx, left);
    }
  }
  // rows whose codes and values this lane writes
  const int rows = whole ? ROW_STEPS : static_cast<int>(min((p.rows - row0 + 31) / 32, int64_t{4}));
  const int written = whole || c < (p.cols + 31) / 32 * 32 ? rows : 0;
  const int64_t step = 32 * p.ldd;
#pragma unroll
  for (int i = 0; i < ROW_STEPS; ++i) {
    float v[8];
    raw[i].get(v);
    uint32_t amax = __float_as_uint(max_abs8(v));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t code = scale_code(amax);
    const uint32_t codes = code == 255u ? 0u : encode8(v, scale_inverse(code));
    codes4 |= code << (8 * i);
    if (i < written) *reinterpret_cast<uint32_t*>(data) = codes;
    data += step;
    if (VALUES && i < rows) {
      decode8(codes, scale_value(code), v);
      Raw8<T> out;
      out.set(v);
      T* dst = static_cast<T*>(p.values) + (row0 + 32 * i) * p.ldv + c;
      if (whole || (VEC && c + 8 <= p.cols))
        out.store(dst);
      else
        out.store(dst, p.cols - c);
    }
  }
  // Of each four blocks (16 lanes) and rows: from a block's bytes in its lanes to a
  // row's in them, by exchanges with the lanes of the next block and the next two.
  uint32_t other = __shfl_xor_sync(0xffffffffu, codes4, 4);
  codes4 = __byte_perm(codes4, other, lane & 4 ? 0x3715 : 0x6240);
  other = __shfl_xor_sync(0xffffffffu, codes4, 8);
  codes4 = __byte_perm(codes4, other, lane & 8 ? 0x3276 : 0x5410);
  if ((lane & 3) == 0 && c / 128 < p.kt)
    *reinterpret_cast<uint32_t*>(p.scales + scale_offset(row0, 0, p.kt) + c / 128 * 512 +
                                 (lane >> 2 & 3) * 4) = codes4;
}

struct ColParams {
  const void* x;
  int64_t ldx, rows, cols;  // of X: blocks run along `rows`
  uint8_t* data;
  int64_t ldd;
  uint8_t* scales;
  void* values;
  int64_t ldv;
  int64_t kt;
  int64_t tiles_n;  // CTAs along X's columns
};

// Blocks down the columns: one pass, bound by HBM.  A warp takes one block of 32
// rows x 32 lanes of columns (one fp32 column a lane, or two 16-bit ones: 128 bytes
// a row either way), so a block's values, maximum and codes all stay in one thread;
// eight warps take eight blocks, and the codes go out through shared memory as 128
// contiguous bytes a packed row.  GB300: 8192 x 11008 fp32 with values 114.7 us (6.7
// TB/s), 8192 x 8192 bf16 27.0 (6.3 TB/s), with values 50.0 (6.1 TB/s).
template <typename T, bool VEC, bool VALUES>
__global__ void __launch_bounds__(256) quantize_cols_kernel(const ColParams p) {
  constexpr int CPT = 4 / sizeof(T);  // columns a thread
  constexpr int COLS = 32 * CPT;
  __shared__ uint4 codes_s[COLS][9];   // 8 blocks a column, padded against bank conflicts
  __shared__ alignas(8) uint8_t scale_s[COLS][8];
  start_in_order();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t tn = static_cast<uint32_t>(p.tiles_n);
  const int64_t ty = blockIdx.x / tn;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x - ty * tn) * COLS;
  const int64_t block = ty * 8 + warp;
  const int64_t k0 = block * 32, n = n0 + lane * CPT;
  // 32 rows of one fp32 value or of two 16-bit ones, as words; a whole block's
  // loads in one go
  const T* src = static_cast<const T*>(p.x) + k0 * p.ldx + n;
  const bool whole = VEC && k0 + 32 <= p.rows && n0 + COLS <= p.cols;
  uint32_t raw[32];
  if (whole) {
#pragma unroll
    for (int i = 0; i < 32; ++i) raw[i] = __ldcs(reinterpret_cast<const uint32_t*>(src + i * p.ldx));
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      alignas(4) T t[CPT];
#pragma unroll
      for (int j = 0; j < CPT; ++j)
        t[j] = k0 + i < p.rows && n + j < p.cols ? src[i * p.ldx + j] : from_float<T>(0.f);
      raw[i] = *reinterpret_cast<const uint32_t*>(t);
    }
  }
  auto value = [&](int i, int j) { return to_float(reinterpret_cast<const T*>(&raw[i])[j]); };
  uint32_t code[CPT], packed[CPT][4];
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 32; i += 2) amax = max_abs3(amax, value(i, j), value(i + 1, j));
    code[j] = scale_code(__float_as_uint(amax));
    const float inv = scale_inverse(code[j]);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = value(8 * g + i, j);
      packed[j][g] = code[j] == 255u ? 0u : encode8(f, inv);
    }
    codes_s[lane * CPT + j][warp] =
        make_uint4(packed[j][0], packed[j][1], packed[j][2], packed[j][3]);
    scale_s[lane * CPT + j][warp] = static_cast<uint8_t>(code[j]);
  }
  if (VALUES) {
    T* dst = static_cast<T*>(p.values) + k0 * p.ldv + n;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float f[CPT][8];
#pragma unroll
      for (int j = 0; j < CPT; ++j) decode8(packed[j][g], scale_value(code[j]), f[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        alignas(4) T t[CPT];
#pragma unroll
        for (int j = 0; j < CPT; ++j) t[j] = from_float<T>(f[j][i]);
        T* at = dst + (8 * g + i) * p.ldv;
        if (whole) {
          *reinterpret_cast<uint32_t*>(at) = *reinterpret_cast<const uint32_t*>(t);
        } else {
#pragma unroll
          for (int j = 0; j < CPT; ++j)
            if (k0 + 8 * g + i < p.rows && n + j < p.cols) at[j] = t[j];
        }
      }
    }
  }
  __syncthreads();
  const int64_t blocks = (p.rows + 31) / 32;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = i * 32 + (threadIdx.x >> 3), part = threadIdx.x & 7;
    if (n0 + c < p.cols && ty * 8 + part < blocks)
      *reinterpret_cast<uint4*>(p.data + (n0 + c) * p.ldd + (ty * 8 + part) * 16) =
          codes_s[c][part];
  }
  if (threadIdx.x < 2 * COLS) {
    const int c = threadIdx.x >> 1, half = threadIdx.x & 1;
    const int64_t tile = ty * 2 + half;
    if (tile < p.kt)
      *reinterpret_cast<uint32_t*>(p.scales + scale_offset(n0 + c, tile * 4, p.kt)) =
          *reinterpret_cast<const uint32_t*>(&scale_s[c][half * 4]);
  }
}

template <typename P>
cudaError_t launch(void (*kern)(P), dim3 grid, const P& p, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
bool vec_ok(const void* p, int64_t ld, int64_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 &&
         ld * static_cast<int64_t>(sizeof(T)) % bytes == 0;
}

template <typename T>
cudaError_t launch_t(const void* X, int64_t rows, int64_t cols, int64_t ldx, bool transpose,
                     uint8_t* data, int64_t ldd, uint8_t* scales, void* values, int64_t ldv,
                     cudaStream_t s) {
  note_launch();
  if (!transpose) {
    const RowParams p{X,      ldx, rows, cols, data, ldd, scales, values, ldv, scale_tiles(cols),
                      static_cast<uint32_t>((scale_tiles(cols) + 1) / 2)};
    const int64_t tasks = (rows + 127) / 128 * 32 * p.chunks;
    if (tasks + 8 > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>((tasks + 7) / 8));
    const bool vec = vec_ok<T>(X, ldx, 16) && (!values || vec_ok<T>(values, ldv, 16));
    auto kern = vec ? (values ? quantize_rows_kernel<T, true, true>
                              : quantize_rows_kernel<T, true, false>)
                    : (values ? quantize_rows_kernel<T, false, true>
                              : quantize_rows_kernel<T, false, false>);
    return launch(kern, grid, p, s);
  }
  constexpr int64_t COLS = 32 * 4 / sizeof(T);
  const ColParams p{X,    ldx,    rows,   cols, data,
                    ldd,  scales, values, ldv,  scale_tiles(rows),
                    (cols + 127) / 128 * 128 / COLS};
  const int64_t ctas = p.tiles_n * ((p.kt + 1) / 2);
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const bool vec = vec_ok<T>(X, ldx, 4) && (!values || vec_ok<T>(values, ldv, 4));
  auto kern = vec ? (values ? quantize_cols_kernel<T, true, true>
                            : quantize_cols_kernel<T, true, false>)
                  : (values ? quantize_cols_kernel<T, false, true>
                            : quantize_cols_kernel<T, false, false>);
  return launch(kern, dim3(static_cast<unsigned>(ctas)), p, s);
}

}  // namespace

cudaError_t launch_quantize(int dtype, const void* X, int64_t rows, int64_t cols, int64_t ldx,
                            bool transpose, uint8_t* data, int64_t ldd, uint8_t* scales,
                            void* values, int64_t ldv, cudaStream_t s) {
  switch (dtype) {
    case MHR_F32:
      return launch_t<float>(X, rows, cols, ldx, transpose, data, ldd, scales, values, ldv, s);
    case MHR_BF16:
      return launch_t<__nv_bfloat16>(X, rows, cols, ldx, transpose, data, ldd, scales, values,
                                     ldv, s);
    default:
      return launch_t<__half>(X, rows, cols, ldx, transpose, data, ldd, scales, values, ldv, s);
  }
}

}  // namespace mx
}  // namespace mhr
