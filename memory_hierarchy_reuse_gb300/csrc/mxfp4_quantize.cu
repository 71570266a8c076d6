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

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// 8 codes in a word, column i in bits [4 i, 4 i + 4).
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], float inv) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i] * inv;
  return e2m1x8(y);
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

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int64_t left, float (&v)[8]) {
  if (VEC && left >= 8) {
    alignas(16) T t[8];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(t) / 16); ++i)
      reinterpret_cast<uint4*>(t)[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_float(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? to_float(p[i]) : 0.f;
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int64_t left, const float (&v)[8]) {
  if (VEC && left >= 8) {
    alignas(16) T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = from_float<T>(v[i]);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(t) / 16); ++i)
      reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(t)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = from_float<T>(v[i]);
  }
}

struct RowParams {
  const void* x;
  int64_t ldx, rows, cols;
  uint8_t* data;
  int64_t ldd;
  uint8_t* scales;
  void* values;
  int64_t ldv;
  int64_t kt;     // scale tiles along a row
  int64_t spans;  // warps along a row
};

constexpr int ROW_CHUNK = 256;  // columns of a warp's step: 8 a lane
constexpr int ROW_STEPS = 4;    // steps a warp has in flight at once
constexpr int ROW_SPAN = ROW_CHUNK * ROW_STEPS;

// Blocks along the rows.  A warp takes 1024 columns of a row in four steps of
// 8 columns a lane (16 bytes of a 16-bit type), all loads first; a block is
// four neighbouring lanes, its maximum two shuffles.  Rows past the last up to
// a multiple of 128 get zero scales (the tiles are written whole).
template <typename T, bool VEC, bool VALUES>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const RowParams p) {
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t task = blockIdx.x * int64_t{8} + (threadIdx.x >> 5);
  const int64_t row = task / p.spans;
  if (row >= (p.rows + 127) / 128 * 128) return;
  const int64_t span0 = (task - row * p.spans) * ROW_SPAN;
  uint8_t* srow = p.scales + scale_offset(row, 0, p.kt);
  if (row >= p.rows) {
    if ((lane & 15) == 0)
      for (int i = 0; i < ROW_STEPS; ++i) {
        const int64_t tile = (span0 + i * ROW_CHUNK + lane * 8) / 128;
        if (tile < p.kt) *reinterpret_cast<uint32_t*>(srow + tile * 512) = 0u;
      }
    return;
  }
  const T* xrow = static_cast<const T*>(p.x) + row * p.ldx;
  float v[ROW_STEPS][8];
#pragma unroll
  for (int i = 0; i < ROW_STEPS; ++i) {
    const int64_t c = span0 + i * ROW_CHUNK + lane * 8;
    if (c < p.cols)
      load8<T, VEC>(xrow + c, p.cols - c, v[i]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < ROW_STEPS; ++i) {
    const int64_t c = span0 + i * ROW_CHUNK + lane * 8;
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, abs_bits(v[i][j]));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t code = scale_code(amax);
    const uint32_t codes = code == 255u ? 0u : encode8(v[i], scale_inverse(code));
    if (c < (p.cols + 31) / 32 * 32)
      *reinterpret_cast<uint32_t*>(p.data + row * p.ldd + c / 2) = codes;
    // the scales of 4 blocks (16 lanes) as one word
    uint32_t word = code << (8 * ((lane >> 2) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if ((lane & 15) == 0 && c / 128 < p.kt)
      *reinterpret_cast<uint32_t*>(srow + c / 128 * 512) = word;
    if (VALUES && c < p.cols) {
      float w[8];
      decode8(codes, scale_value(code), w);
      store8<T, VEC>(static_cast<T*>(p.values) + row * p.ldv + c, p.cols - c, w);
    }
  }
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

// Blocks down the columns.  A warp takes one block of 32 rows x 32 lanes of
// columns (one fp32 column a lane, or two 16-bit ones: 128 bytes a row either
// way), so a block's values, maximum and codes all stay in one thread; eight
// warps take eight blocks, and the codes go out through shared memory as 128
// contiguous bytes a packed row.
template <typename T, bool VEC, bool VALUES>
__global__ void __launch_bounds__(256) quantize_cols_kernel(const ColParams p) {
  constexpr int CPT = 4 / sizeof(T);  // columns a thread
  constexpr int COLS = 32 * CPT;
  __shared__ uint4 codes_s[COLS][9];   // 8 blocks a column, padded against bank conflicts
  __shared__ alignas(8) uint8_t scale_s[COLS][8];
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t ty = blockIdx.x / p.tiles_n;
  const int64_t n0 = (blockIdx.x - ty * p.tiles_n) * COLS;
  const int64_t block = ty * 8 + warp;
  const int64_t k0 = block * 32, n = n0 + lane * CPT;
  const T* x = static_cast<const T*>(p.x);
  T v[32][CPT];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const int64_t k = k0 + i;
    const T* src = x + k * p.ldx + n;
    if (VEC && CPT == 2 && k < p.rows && n + 1 < p.cols) {
      *reinterpret_cast<uint32_t*>(v[i]) = __ldcs(reinterpret_cast<const uint32_t*>(src));
    } else {
#pragma unroll
      for (int j = 0; j < CPT; ++j)
        v[i][j] = k < p.rows && n + j < p.cols ? src[j] : from_float<T>(0.f);
    }
  }
  float scale[CPT];
  uint4 packed[CPT];
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = max(amax, abs_bits(to_float(v[i][j])));
    const uint32_t code = scale_code(amax);
    const float inv = scale_inverse(code);
    scale[j] = scale_value(code);
    uint32_t w[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = to_float(v[8 * g + i][j]);
      w[g] = code == 255u ? 0u : encode8(f, inv);
    }
    packed[j] = make_uint4(w[0], w[1], w[2], w[3]);
    codes_s[lane * CPT + j][warp] = packed[j];
    scale_s[lane * CPT + j][warp] = static_cast<uint8_t>(code);
  }
  if (VALUES) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float f[CPT][8];
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        const uint32_t w = g == 0   ? packed[j].x
                           : g == 1 ? packed[j].y
                           : g == 2 ? packed[j].z
                                    : packed[j].w;
        decode8(w, scale[j], f[j]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t k = k0 + 8 * g + i;
        if (k >= p.rows) break;
        T* dst = static_cast<T*>(p.values) + k * p.ldv + n;
        if (VEC && CPT == 2 && n + 1 < p.cols) {
          T t[2] = {from_float<T>(f[0][i]), from_float<T>(f[CPT - 1][i])};
          *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(t);
        } else {
#pragma unroll
          for (int j = 0; j < CPT; ++j)
            if (n + j < p.cols) dst[j] = from_float<T>(f[j][i]);
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
                      (scale_tiles(cols) * 128 + ROW_SPAN - 1) / ROW_SPAN};
    const int64_t tasks = (rows + 127) / 128 * 128 * p.spans;
    if ((tasks + 7) / 8 > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>((tasks + 7) / 8));
    const bool vec = vec_ok<T>(X, ldx, 16) && (!values || vec_ok<T>(values, ldv, 16));
    auto kern = vec ? (values ? quantize_rows_kernel<T, true, true>
                              : quantize_rows_kernel<T, true, false>)
                    : (values ? quantize_rows_kernel<T, false, true>
                              : quantize_rows_kernel<T, false, false>);
    kern<<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
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
  kern<<<dim3(static_cast<unsigned>(ctas)), 256, 0, s>>>(p);
  return cudaGetLastError();
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
