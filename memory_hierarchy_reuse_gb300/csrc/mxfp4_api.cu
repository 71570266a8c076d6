// C-ABI front end of the 4-bit operators (include/mhr_mxfp4.h): argument
// checks, workspaces and dispatch.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "mhr_gemm.h"
#include "mhr_mxfp4.h"
#include "mxfp4_internal.h"

#define MHR_API extern "C" __attribute__((visibility("default")))

namespace mhr {
namespace mx {
namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 512;  // tile/TMA coordinates are int32

int from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return MHR_OK;
  cudaGetLastError();
  return MHR_ERR_CUDA;
}

bool dims_ok(int64_t a, int64_t b) { return a >= 0 && b >= 0 && a <= kMaxDim && b <= kMaxDim; }
bool dtype_ok(int d) { return d == MHR_F32 || d == MHR_BF16 || d == MHR_F16; }
int64_t size_of(int dtype) { return dtype == MHR_F32 ? 4 : 2; }
bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A plain matrix of `dtype`: pointer, pitch and alignment to its elements.
bool plain_ok(int dtype, const void* p, int64_t rows, int64_t cols, int64_t ld, ByteRange* r) {
  const int64_t size = size_of(dtype);
  int64_t pitch;
  return p && ld >= cols && aligned(p, size) && !__builtin_mul_overflow(ld, size, &pitch) &&
         byte_range(p, rows, cols * size, pitch, r);
}

// A packed matrix: its two arrays, aligned for 16-byte and TMA access.
bool packed_ok(const uint8_t* data, const uint8_t* scales, int64_t rows, int64_t cols, int64_t ld,
               ByteRange* rd, ByteRange* rs) {
  const int64_t row_bytes = blocks_of(cols) * 16;
  return data && scales && aligned(data, 16) && aligned(scales, 16) && ld % 16 == 0 &&
         ld >= row_bytes && ld < (int64_t{1} << 40) && byte_range(data, rows, row_bytes, ld, rd) &&
         byte_range(scales, 1, scale_bytes(rows, cols), scale_bytes(rows, cols), rs);
}

// C and B^T of a product, and their being apart; K > 0.
int check_product(int c_dtype, const uint8_t* Bt, const uint8_t* Bt_scales, const void* C,
                  int64_t M, int64_t N, int64_t K, int64_t ldb, int64_t ldc, ByteRange* rc) {
  ByteRange rb, rsb;
  if (!plain_ok(c_dtype, C, M, N, ldc, rc)) return MHR_ERR_INVALID_ARG;
  if (K == 0) return MHR_OK;
  if (!packed_ok(Bt, Bt_scales, N, K, ldb, &rb, &rsb)) return MHR_ERR_INVALID_ARG;
  if (ranges_overlap(*rc, rb) || ranges_overlap(*rc, rsb)) return MHR_ERR_INVALID_ARG;
  return MHR_OK;
}

// C = 0 (K == 0): zero bytes are zero in every type.
cudaError_t zero_c(int c_dtype, void* C, int64_t M, int64_t N, int64_t ldc, cudaStream_t s) {
  const int64_t size = size_of(c_dtype);
  return cudaMemset2DAsync(C, static_cast<size_t>(ldc * size), 0, static_cast<size_t>(N * size),
                           static_cast<size_t>(M), s);
}

// Up to 32 rows the narrow kernel runs, two CTAs an SM (GB300, narrow against
// pair: 32 x 4096 x 4096 6.9 / 8.8 us, 32 x 28672 x 4096 13.7 / 19.1); more by the
// two kernels' estimates (64 x 4096 x 4096 7.4 / 8.9, 64 x 28672 x 4096 20.7 /
// 16.4; 200 x 300 x 8192 7.8 / 13.5, 200 x 4096 x 4096 11.8 / 9.1).
// gemm_testing_set_cta_pair_mode picks a kernel, as for the other products.
cudaError_t launch_product(const ProductArgs& a, const DeviceCtl& ctl, int device,
                           cudaStream_t s) {
  bool pair = ctl.pair_mode == 2;
  if (ctl.pair_mode == 0 && a.M > 32) {
    double narrow = 0;
    const cudaError_t e = narrow_time(a.M, a.N, a.K, ctl.sm_count, device, &narrow);
    if (e != cudaSuccess) return e;
    pair = pair_time(a.M, a.N, a.K, ctl.sm_count / 2) < narrow;
  }
  MainKernelEvents ev(s);
  return pair ? launch_pair(a, ctl, s) : launch_narrow(a, ctl, s);
}

}  // namespace
}  // namespace mx
}  // namespace mhr

using namespace mhr;
using namespace mhr::mx;

MHR_API int64_t gemm_mxfp4_scale_bytes(int64_t rows, int64_t cols) {
  return dims_ok(rows, cols) ? scale_bytes(rows, cols) : -1;
}

MHR_API int gemm_mxfp4_quantize(int dtype, const void* X, int64_t rows, int64_t cols, int64_t ldx,
                                int transpose, uint8_t* data, int64_t ldd, uint8_t* scales,
                                void* values, int64_t ldv, void* stream) {
  if (!dtype_ok(dtype) || !dims_ok(rows, cols)) return MHR_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return MHR_OK;
  ByteRange rx, rd, rs, rv;
  const int64_t prows = transpose ? cols : rows, pcols = transpose ? rows : cols;
  if (!plain_ok(dtype, X, rows, cols, ldx, &rx) ||
      !packed_ok(data, scales, prows, pcols, ldd, &rd, &rs) ||
      (values && !plain_ok(dtype, values, rows, cols, ldv, &rv)))
    return MHR_ERR_INVALID_ARG;
  if (ranges_overlap(rx, rd) || ranges_overlap(rx, rs) || ranges_overlap(rx, rv) ||
      ranges_overlap(rd, rs) || ranges_overlap(rd, rv) || ranges_overlap(rs, rv))
    return MHR_ERR_INVALID_ARG;
  begin_call();
  std::lock_guard<std::mutex> lock(library_mutex());
  DeviceCtl ctl;
  int dev = 0;
  if (const int rc = device_ctl_locked(&ctl, &dev); rc != MHR_OK) return rc;
  return from_cuda(launch_quantize(dtype, X, rows, cols, ldx, transpose != 0, data, ldd, scales,
                                   values, ldv, static_cast<cudaStream_t>(stream)));
}

MHR_API int gemm_mxfp4(int c_dtype, const uint8_t* A, const uint8_t* A_scales, const uint8_t* Bt,
                       const uint8_t* Bt_scales, void* C, int64_t M, int64_t N, int64_t K,
                       int64_t lda, int64_t ldb, int64_t ldc, void* stream) {
  if (!dtype_ok(c_dtype) || !dims_ok(M, N) || !dims_ok(K, 0)) return MHR_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return MHR_OK;
  ByteRange rc, ra, rsa;
  if (const int st = check_product(c_dtype, Bt, Bt_scales, C, M, N, K, ldb, ldc, &rc);
      st != MHR_OK)
    return st;
  if (K > 0 && (!packed_ok(A, A_scales, M, K, lda, &ra, &rsa) || ranges_overlap(rc, ra) ||
                ranges_overlap(rc, rsa)))
    return MHR_ERR_INVALID_ARG;
  begin_call();
  std::lock_guard<std::mutex> lock(library_mutex());
  DeviceCtl ctl;
  int dev = 0;
  if (const int st = device_ctl_locked(&ctl, &dev); st != MHR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) return from_cuda(zero_c(c_dtype, C, M, N, ldc, s));
  return from_cuda(launch_product(
      {A, A_scales, lda, Bt, Bt_scales, ldb, C, ldc, c_dtype, M, N, K, false}, ctl, dev, s));
}

MHR_API int gemm_mxfp4_quantized(int a_dtype, const void* A, int c_dtype, const uint8_t* Bt,
                                 const uint8_t* Bt_scales, void* C, int64_t M, int64_t N,
                                 int64_t K, int64_t lda, int64_t ldb, int64_t ldc, void* stream) {
  if (!dtype_ok(a_dtype) || !dtype_ok(c_dtype) || !dims_ok(M, N) || !dims_ok(K, 0))
    return MHR_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return MHR_OK;
  ByteRange rc, ra;
  if (const int st = check_product(c_dtype, Bt, Bt_scales, C, M, N, K, ldb, ldc, &rc);
      st != MHR_OK)
    return st;
  if (K > 0 && (!plain_ok(a_dtype, A, M, K, lda, &ra) || ranges_overlap(rc, ra)))
    return MHR_ERR_INVALID_ARG;
  begin_call();
  std::lock_guard<std::mutex> lock(library_mutex());
  DeviceCtl ctl;
  int dev = 0;
  if (const int st = device_ctl_locked(&ctl, &dev); st != MHR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) return from_cuda(zero_c(c_dtype, C, M, N, ldc, s));
  bool fused = false;
  if (ctl.pair_mode != 2)
    if (const cudaError_t e = narrow_quantizes(M, N, K, a_dtype, dev, &fused); e != cudaSuccess)
      return from_cuda(e);
  if (fused) {
    ProductArgs a{nullptr, nullptr, lda, Bt, Bt_scales, ldb, C, ldc, c_dtype, M, N, K};
    a.a_plain = A;
    a.a_dtype = a_dtype;
    return from_cuda(launch_product(a, ctl, dev, s));
  }
  const int64_t row_bytes = blocks_of(K) * 16;
  size_t data_bytes;
  if (__builtin_mul_overflow(static_cast<size_t>(M), static_cast<size_t>(row_bytes), &data_bytes))
    return MHR_ERR_CUDA;
  void *ws, *token;
  if (const int st = workspace_locked(dev, s, data_bytes + scale_bytes(M, K), &ws, &token);
      st != MHR_OK)
    return st;
  uint8_t* data = static_cast<uint8_t*>(ws);
  uint8_t* scales = data + data_bytes;
  cudaError_t e =
      launch_quantize(a_dtype, A, M, K, lda, false, data, row_bytes, scales, nullptr, 0, s);
  if (e == cudaSuccess)
    e = launch_product(
        {data, scales, row_bytes, Bt, Bt_scales, ldb, C, ldc, c_dtype, M, N, K, true}, ctl, dev, s);
  workspace_done_locked(token, s);
  return from_cuda(e);
}

MHR_API int gemm_mxfp4_moe(const uint16_t* x, int64_t ldx, const uint16_t* router, int64_t ldr,
                           const uint8_t* up, const uint8_t* up_scales, int64_t ldu,
                           const uint8_t* down, const uint8_t* down_scales, int64_t ldd,
                           uint16_t* y, int64_t ldy, int32_t* experts, float* weights, int64_t T,
                           int64_t E, int64_t top, int64_t H, int64_t I, void* stream) {
  static_assert(MOE_CONTROL_BYTES <= kControlBytes, "the layer's counters");
  if (T < 0 || T > MOE_MAX_TOKENS || E < 1 || E > MOE_MAX_EXPERTS || top < 1 ||
      top > MOE_MAX_TOP || top > E || H < 1 || H > MOE_MAX_WIDTH || I < 1 || I > MOE_MAX_WIDTH)
    return MHR_ERR_INVALID_ARG;
  if (T == 0) return MHR_OK;
  ByteRange in[6], out[3];
  if (!plain_ok(MHR_BF16, x, T, H, ldx, &in[0]) ||
      !plain_ok(MHR_BF16, router, E, H, ldr, &in[1]) ||
      !packed_ok(up, up_scales, 2 * E * I, H, ldu, &in[2], &in[3]) ||
      !packed_ok(down, down_scales, E * H, I, ldd, &in[4], &in[5]) ||
      !plain_ok(MHR_BF16, y, T, H, ldy, &out[0]) ||
      !plain_ok(MHR_F32, experts, 1, T * top, T * top, &out[1]) ||
      !plain_ok(MHR_F32, weights, 1, T * top, T * top, &out[2]))
    return MHR_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    for (const ByteRange& r : in)
      if (ranges_overlap(out[i], r)) return MHR_ERR_INVALID_ARG;
    if (ranges_overlap(out[i], out[(i + 1) % 3])) return MHR_ERR_INVALID_ARG;
  }
  begin_call();
  std::lock_guard<std::mutex> lock(library_mutex());
  DeviceCtl ctl;
  int dev = 0;
  if (const int st = device_ctl_locked(&ctl, &dev); st != MHR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const MoeArgs a{x,    ldx,         router, ldr, up, up_scales, ldu, down,
                  down_scales, ldd,  y,      ldy, experts, weights, T, E, top, H, I};
  size_t at[5];
  void *ws, *token, *control;
  if (const int st = workspace_locked(dev, s, moe_workspace(a, at), &ws, &token); st != MHR_OK)
    return st;
  if (const int st = workspace_control_locked(token, s, &control); st != MHR_OK) return st;
  cudaError_t e;
  {
    MainKernelEvents ev(s);
    e = launch_moe(a, ws, static_cast<uint32_t*>(control), ctl, s);
  }
  workspace_done_locked(token, s);
  return from_cuda(e);
}
