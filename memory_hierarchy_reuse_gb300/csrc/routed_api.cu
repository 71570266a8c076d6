// C-ABI front end of the operators that go by an index per row
// (include/mhr_routed.h): argument checks and dispatch.
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <mutex>

#include "mhr_gemm.h"
#include "mhr_routed.h"
#include "routed_internal.h"

#define MHR_API extern "C" __attribute__((visibility("default")))

namespace mhr {
namespace routed {
namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 512;  // row and column numbers are int32

int from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return MHR_OK;
  cudaGetLastError();
  return MHR_ERR_CUDA;
}

bool dim_ok(int64_t n) { return n >= 0 && n <= kMaxDim; }
bool dtype_ok(int d) { return d == MHR_F32 || d == MHR_BF16 || d == MHR_F16; }
int64_t size_of(int dtype) { return dtype == MHR_F32 ? 4 : 2; }
bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A plain matrix of elements of `size` bytes: pointer, pitch and alignment.
bool plain_ok(const void* p, int64_t size, int64_t rows, int64_t cols, int64_t ld, ByteRange* r) {
  int64_t pitch;
  return p && ld >= cols && aligned(p, size) && !__builtin_mul_overflow(ld, size, &pitch) &&
         byte_range(p, rows, cols * size, pitch, r);
}
bool array_ok(const void* p, int64_t size, int64_t n, ByteRange* r) {
  return plain_ok(p, size, 1, n, n, r);
}

bool apart(std::initializer_list<ByteRange> out, std::initializer_list<ByteRange> in) {
  for (auto o = out.begin(); o != out.end(); ++o) {
    for (const ByteRange& i : in)
      if (ranges_overlap(*o, i)) return false;
    for (auto q = out.begin(); q != o; ++q)
      if (ranges_overlap(*o, *q)) return false;
  }
  return true;
}

// The launch of a validated call on the current device.
template <typename F>
int launched(const F& f) {
  begin_call();
  std::lock_guard<std::mutex> lock(library_mutex());
  DeviceCtl ctl;
  int dev = 0;
  if (const int rc = device_ctl_locked(&ctl, &dev); rc != MHR_OK) return rc;
  return from_cuda(f(ctl));
}

bool router_ok(int64_t T, int64_t E, int64_t top, int score) {
  return dim_ok(T) && E >= 1 && E <= MAX_EXPERTS && top >= 1 && top <= MAX_TOP && top <= E &&
         (score == MHR_SOFTMAX || score == MHR_SIGMOID);
}

// `parts` matrices, `stride` elements apart, that do not reach into one another.
bool parts_ok(const void* p, int64_t size, int64_t parts, int64_t rows, int64_t cols, int64_t ld,
              int64_t stride, ByteRange* r) {
  int64_t all, span, bytes;
  if (parts == 1) return plain_ok(p, size, rows, cols, ld, r);
  ByteRange one;
  return plain_ok(p, size, rows, cols, ld, &one) && !__builtin_mul_overflow(rows - 1, ld, &span) &&
         !__builtin_add_overflow(span, cols, &span) && stride >= span &&
         !__builtin_mul_overflow(stride, size, &bytes) &&
         !__builtin_mul_overflow(parts, bytes, &all) && byte_range(p, parts, span * size, bytes, r);
}

// Scratch of `need` bytes (each operand_bytes, -1 if there is no such).
int scratch_ok(const void* scratch, int64_t have, int64_t need_a, int64_t need_b, ByteRange* r) {
  int64_t need;
  if (need_a < 0 || need_b < 0 || __builtin_add_overflow(need_a, need_b, &need))
    return MHR_ERR_CUDA;
  if (need == 0) return MHR_OK;
  return scratch && aligned(scratch, 16) && have >= need && byte_range(scratch, 1, need, need, r)
             ? MHR_OK
             : MHR_ERR_INVALID_ARG;
}

// What both products ask of the types, the sizes and the indices.
bool indexed_ok(int dtype, int out_dtype, int64_t x_rows, const int32_t* gather, int64_t top,
                int64_t other_rows, const int32_t* scatter, const int32_t* offsets, int64_t E,
                int64_t rows, int64_t K, int64_t N, ByteRange (&r)[3]) {
  return (dtype == MHR_BF16 || dtype == MHR_F16) && dtype_ok(out_dtype) && dim_ok(x_rows) &&
         dim_ok(other_rows) && dim_ok(rows) && dim_ok(K) && dim_ok(N) && E >= 1 &&
         E <= MAX_PARTS && top >= 1 && top <= kMaxDim && (gather || x_rows == rows) &&
         (scatter || other_rows == rows) && array_ok(offsets, 4, E + 1, &r[0]) &&
         (!gather || rows == 0 || array_ok(gather, 4, rows, &r[1])) &&
         (!scatter || rows == 0 || array_ok(scatter, 4, rows, &r[2]));
}

}  // namespace
}  // namespace routed
}  // namespace mhr

using namespace mhr;
using namespace mhr::routed;

MHR_API int gemm_routed_choose(int dtype, const void* logits, int64_t T, int64_t E, int64_t ld,
                               int score, const float* bias, int64_t groups, int64_t group_top,
                               int group_score, int64_t top, int renormalize, float scale,
                               int32_t* experts, float* weights, void* stream) {
  if (!dtype_ok(dtype) || !router_ok(T, E, top, score) || groups < 1 || groups > MAX_GROUPS ||
      E % groups || group_top < 1 || group_top > groups || top > group_top * (E / groups) ||
      (group_score != MHR_GROUP_MAX && group_score != MHR_GROUP_TOP2))
    return MHR_ERR_INVALID_ARG;
  if (T == 0) return MHR_OK;
  ByteRange rl, rb, re, rw;
  if (!plain_ok(logits, size_of(dtype), T, E, ld, &rl) ||
      (bias && !array_ok(bias, 4, E, &rb)) || !array_ok(experts, 4, T * top, &re) ||
      !array_ok(weights, 4, T * top, &rw) || !apart({re, rw}, {rl, rb}))
    return MHR_ERR_INVALID_ARG;
  return launched([&](const DeviceCtl&) {
    return launch_choose({dtype, logits, T, E, ld, score, bias, groups, group_top, group_score,
                          top, renormalize != 0, scale, experts, weights},
                         static_cast<cudaStream_t>(stream));
  });
}

MHR_API int gemm_routed_choose_grad(int dtype, const void* logits, int64_t ld,
                                    const int32_t* experts, const float* grad_weights, int64_t T,
                                    int64_t E, int64_t top, int score, int renormalize,
                                    float scale, void* grad_logits, int64_t ldg, void* stream) {
  if (!dtype_ok(dtype) || !router_ok(T, E, top, score)) return MHR_ERR_INVALID_ARG;
  if (T == 0) return MHR_OK;
  ByteRange rl, re, rw, rg;
  if (!plain_ok(logits, size_of(dtype), T, E, ld, &rl) || !array_ok(experts, 4, T * top, &re) ||
      !array_ok(grad_weights, 4, T * top, &rw) ||
      !plain_ok(grad_logits, size_of(dtype), T, E, ldg, &rg) || !apart({rg}, {rl, re, rw}))
    return MHR_ERR_INVALID_ARG;
  return launched([&](const DeviceCtl&) {
    return launch_choose_grad({dtype, logits, ld, experts, grad_weights, T, E, top, score,
                               renormalize != 0, scale, grad_logits, ldg},
                              static_cast<cudaStream_t>(stream));
  });
}

MHR_API int gemm_routed_sort(const int32_t* experts, int64_t n, int64_t E, int32_t* offsets,
                             int32_t* order, void* stream) {
  if (!dim_ok(n) || E < 1 || E > MAX_PARTS) return MHR_ERR_INVALID_ARG;
  ByteRange re, ro, rr;
  if ((n > 0 && (!array_ok(experts, 4, n, &re) || !array_ok(order, 4, n, &rr))) ||
      !array_ok(offsets, 4, E + 1, &ro) || !apart({ro, rr}, {re}))
    return MHR_ERR_INVALID_ARG;
  return launched([&](const DeviceCtl&) {
    return launch_sort(experts, n, E, offsets, order, static_cast<cudaStream_t>(stream));
  });
}

MHR_API int64_t gemm_routed_product_scratch(const void* x, int64_t x_rows, int64_t ldx,
                                            int gathered, const void* w, int64_t ldw,
                                            int64_t stride_w, int transposed, int64_t E,
                                            int64_t rows, int64_t K, int64_t N) {
  if (E < 1 || E > MAX_PARTS || !dim_ok(x_rows) || !dim_ok(rows) || !dim_ok(K) || !dim_ok(N))
    return -1;
  if (rows == 0 || N == 0 || K == 0 || x_rows == 0) return 0;
  const int64_t a =
      operand_bytes(x, 1, x_rows, K, ldx, 0, gathered && rows > FEW_ROWS ? rows : 0);
  const int64_t b =
      operand_bytes(w, E, transposed ? N : K, transposed ? K : N, ldw, stride_w, 0);
  int64_t both;
  return a < 0 || b < 0 || __builtin_add_overflow(a, b, &both) ? -1 : both;
}

MHR_API int64_t gemm_routed_weight_grad_scratch(const void* x, int64_t x_rows, int64_t ldx,
                                                int gathered, const void* grad,
                                                int64_t grad_rows, int64_t ldg, int scattered,
                                                int64_t rows, int64_t K, int64_t N) {
  if (!dim_ok(x_rows) || !dim_ok(grad_rows) || !dim_ok(rows) || !dim_ok(K) || !dim_ok(N))
    return -1;
  if (rows == 0 || N == 0 || K == 0 || x_rows == 0 || grad_rows == 0) return 0;
  const int64_t a = operand_bytes(x, 1, x_rows, K, ldx, 0, gathered ? rows : 0);
  const int64_t b = operand_bytes(grad, 1, grad_rows, N, ldg, 0, scattered ? rows : 0);
  int64_t both;
  return a < 0 || b < 0 || __builtin_add_overflow(a, b, &both) ? -1 : both;
}

MHR_API int gemm_routed_product(int dtype, const void* x, int64_t x_rows, int64_t ldx,
                                const int32_t* gather, int64_t top, const void* w, int64_t ldw,
                                int64_t stride_w, int transposed, const int32_t* offsets,
                                int64_t E, int out_dtype, void* out, int64_t out_rows,
                                int64_t ldo, const int32_t* scatter, int64_t rows, int64_t K,
                                int64_t N, void* scratch, int64_t scratch_bytes, void* stream) {
  ByteRange index[3], rx, rw, ro, rs;
  if (!indexed_ok(dtype, out_dtype, x_rows, gather, top, out_rows, scatter, offsets, E, rows, K, N,
                  index))
    return MHR_ERR_INVALID_ARG;
  if (rows == 0 || N == 0 || out_rows == 0) return MHR_OK;
  if (!plain_ok(out, size_of(out_dtype), out_rows, N, ldo, &ro)) return MHR_ERR_INVALID_ARG;
  if (K > 0 && x_rows > 0) {
    const int64_t wr = transposed ? N : K, wc = transposed ? K : N;
    if (!plain_ok(x, 2, x_rows, K, ldx, &rx) || !parts_ok(w, 2, E, wr, wc, ldw, stride_w, &rw))
      return MHR_ERR_INVALID_ARG;
    if (const int rc = scratch_ok(
            scratch, scratch_bytes,
            operand_bytes(x, 1, x_rows, K, ldx, 0, gather && rows > FEW_ROWS ? rows : 0),
            operand_bytes(w, E, wr, wc, ldw, stride_w, 0), &rs);
        rc != MHR_OK)
      return rc;
  }
  if (!apart({ro, rs}, {index[0], index[1], index[2], rx, rw})) return MHR_ERR_INVALID_ARG;
  return launched([&](const DeviceCtl& ctl) {
    return launch_product({transposed ? ProductKind::transposed : ProductKind::product, dtype, x,
                           x_rows, ldx, gather, top, w, ldw, stride_w, offsets, E, out_dtype, out,
                           out_rows, ldo, 0, scatter, rows, K, N},
                          scratch, ctl, static_cast<cudaStream_t>(stream));
  });
}

MHR_API int gemm_routed_weight_grad(int dtype, const void* x, int64_t x_rows, int64_t ldx,
                                    const int32_t* gather, int64_t top, const void* grad,
                                    int64_t grad_rows, int64_t ldg, const int32_t* scatter,
                                    const int32_t* offsets, int64_t E, int out_dtype, void* out,
                                    int64_t ldo, int64_t stride_o, int64_t rows, int64_t K,
                                    int64_t N, void* scratch, int64_t scratch_bytes,
                                    void* stream) {
  ByteRange index[3], rx, rg, ro, rs;
  if (!indexed_ok(dtype, out_dtype, x_rows, gather, top, grad_rows, scatter, offsets, E, rows, K,
                  N, index))
    return MHR_ERR_INVALID_ARG;
  if (K == 0 || N == 0) return MHR_OK;
  if (!parts_ok(out, size_of(out_dtype), E, K, N, ldo, stride_o, &ro)) return MHR_ERR_INVALID_ARG;
  if (rows > 0 && x_rows > 0 && grad_rows > 0) {
    if (!plain_ok(x, 2, x_rows, K, ldx, &rx) || !plain_ok(grad, 2, grad_rows, N, ldg, &rg))
      return MHR_ERR_INVALID_ARG;
    if (const int rc = scratch_ok(
            scratch, scratch_bytes, operand_bytes(x, 1, x_rows, K, ldx, 0, gather ? rows : 0),
            operand_bytes(grad, 1, grad_rows, N, ldg, 0, scatter ? rows : 0), &rs);
        rc != MHR_OK)
      return rc;
  }
  if (!apart({ro, rs}, {index[0], index[1], index[2], rx, rg})) return MHR_ERR_INVALID_ARG;
  return launched([&](const DeviceCtl& ctl) {
    return launch_product({ProductKind::gradient, dtype, x, x_rows, ldx, gather, top, grad, ldg, 0,
                           offsets, E, out_dtype, out, grad_rows, ldo, stride_o, scatter, rows, K,
                           N},
                          scratch, ctl, static_cast<cudaStream_t>(stream));
  });
}

namespace {
bool adapters_ok(int dtype, int out_dtype, int64_t L, int64_t rank, int64_t T, int64_t K,
                 int64_t N) {
  return (dtype == MHR_BF16 || dtype == MHR_F16) && dtype_ok(out_dtype) && L >= 1 &&
         L <= MAX_PARTS && rank >= 1 && rank <= MAX_RANK && dim_ok(T) && T <= kMaxDim / 8 &&
         dim_ok(K) && dim_ok(N);
}
}  // namespace

MHR_API int64_t gemm_routed_adapters_scratch(int dtype, const void* x, int64_t ldx,
                                             const void* down, int64_t ldd, int64_t stride_d,
                                             const void* up, int64_t ldu, int64_t stride_u,
                                             int64_t L, int64_t rank, int out_dtype, int64_t T,
                                             int64_t K, int64_t N) {
  if (!adapters_ok(dtype, out_dtype, L, rank, T, K, N)) return -1;
  if (T == 0 || N == 0) return 0;
  return adapters_scratch({dtype, x, ldx, down, ldd, stride_d, up, ldu, stride_u, nullptr, nullptr,
                           L, rank, out_dtype, nullptr, 0, nullptr, 0, T, K, N});
}

MHR_API int gemm_routed_adapters(int dtype, const void* x, int64_t ldx, const void* down,
                                 int64_t ldd, int64_t stride_d, const void* up, int64_t ldu,
                                 int64_t stride_u, const int32_t* which, const float* scales,
                                 int64_t L, int64_t rank, int out_dtype, const void* y,
                                 int64_t ldy, void* out, int64_t ldo, int64_t T, int64_t K,
                                 int64_t N, void* scratch, int64_t scratch_bytes, void* stream) {
  if (!adapters_ok(dtype, out_dtype, L, rank, T, K, N)) return MHR_ERR_INVALID_ARG;
  if (T == 0 || N == 0) return MHR_OK;
  ByteRange rx, rd, ru, rw, rc, ry, ro, rs;
  const int64_t size = size_of(out_dtype);
  if (!plain_ok(y, size, T, N, ldy, &ry) || !plain_ok(out, size, T, N, ldo, &ro) ||
      !array_ok(which, 4, T, &rw) || (scales && !array_ok(scales, 4, L, &rc)) ||
      (K > 0 && (!plain_ok(x, 2, T, K, ldx, &rx) ||
                 !parts_ok(down, 2, L, rank, K, ldd, stride_d, &rd))) ||
      !parts_ok(up, 2, L, rank, N, ldu, stride_u, &ru))
    return MHR_ERR_INVALID_ARG;
  const AdapterArgs a{dtype, x, ldx, down, ldd, stride_d, up, ldu, stride_u, which, scales, L,
                      rank, out_dtype, y, ldy, out, ldo, T, K, N};
  if (const int rc2 = scratch_ok(scratch, scratch_bytes, adapters_scratch(a), 0, &rs);
      rc2 != MHR_OK)
    return rc2;
  if (out == y && (ldo == ldy || T == 1)) ry = ByteRange{};  // in place
  if (!apart({ro, rs}, {rx, rd, ru, rw, rc, ry})) return MHR_ERR_INVALID_ARG;
  return launched([&](const DeviceCtl& ctl) {
    return launch_adapters(a, scratch, ctl, static_cast<cudaStream_t>(stream));
  });
}
