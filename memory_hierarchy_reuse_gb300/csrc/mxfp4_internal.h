// Launchers of the 4-bit operators, shared between their C-ABI front end
// (mxfp4_api.cu) and their kernels.  As in mhr_internal.h, launchers assume
// validated arguments (sizes >= 1, pointers non-null) and return the launch's
// cudaError_t.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "mhr_internal.h"

namespace mhr {
namespace mx {

inline int64_t blocks_of(int64_t cols) { return (cols + 31) / 32; }
// Tiles of 4 blocks along a row of scales.
inline int64_t scale_tiles(int64_t cols) { return (blocks_of(cols) + 3) / 4; }
inline int64_t scale_bytes(int64_t rows, int64_t cols) {
  return (rows + 127) / 128 * scale_tiles(cols) * 512;
}

// X (rows x cols, pitch ldx elements) of type dtype (mhr_dtype) -> codes and
// scales.  transpose: blocks run down X's columns and the packed matrix is
// X^T.  values (or null): what the codes stand for, X's type and shape, pitch
// ldv.
cudaError_t launch_quantize(int dtype, const void* X, int64_t rows, int64_t cols, int64_t ldx,
                            bool transpose, uint8_t* data, int64_t ldd, uint8_t* scales,
                            void* values, int64_t ldv, cudaStream_t s);

// One product C = A B with both operands packed (B as B^T).
struct ProductArgs {
  const uint8_t* A;
  const uint8_t* sfa;
  int64_t lda;
  const uint8_t* B;
  const uint8_t* sfb;
  int64_t ldb;
  void* C;
  int64_t ldc;
  int c_dtype;
  int64_t M, N, K;
  // A was quantised by a kernel of the same call just before, itself launched
  // in plain stream order: B is complete once this kernel starts.
  bool after_quantize;
};
// Few rows of A (any M is right).
cudaError_t launch_narrow(const ProductArgs& a, const DeviceCtl& ctl, cudaStream_t s);

}  // namespace mx
}  // namespace mhr
