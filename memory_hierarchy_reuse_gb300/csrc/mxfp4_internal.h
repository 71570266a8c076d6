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
  // A was quantised by a kernel of the same call just before, which lets this
  // one start only after everything before it: B is complete then.
  bool after_quantize = false;
  // launch_narrow only, where narrow_quantizes: A as a plain matrix (pitch lda
  // elements) instead of packed.
  const void* a_plain = nullptr;
  int a_dtype = 0;
};
// Whether launch_narrow takes a plain A and quantises it on the way: at most
// 32 rows whose part of K fits beside the ring and is little work.
cudaError_t narrow_quantizes(int64_t M, int64_t N, int64_t K, int a_dtype, int device, bool* yes);
// What either kernel takes for a product of packed operands, in us: fits of the
// times measured on GB300, for the choice between the two.
cudaError_t narrow_time(int64_t M, int64_t N, int64_t K, int sms, int device, double* us);
double pair_time(int64_t M, int64_t N, int64_t K, int clusters);
// Few rows of A (any M is right).
cudaError_t launch_narrow(const ProductArgs& a, const DeviceCtl& ctl, cudaStream_t s);
// Many rows of A: CTA pairs on 256 x 256 tiles (any M is right).
cudaError_t launch_pair(const ProductArgs& a, const DeviceCtl& ctl, cudaStream_t s);

// One mixture-of-experts layer (gemm_mxfp4_moe).
constexpr int MOE_MAX_TOKENS = 64, MOE_MAX_TOP = 16, MOE_MAX_EXPERTS = 512;
constexpr int64_t MOE_MAX_WIDTH = 16384;  // H and I
// Counters that a call needs zeroed and leaves zeroed: barrier arrivals, exits.
constexpr size_t MOE_CONTROL_BYTES = 2 * 4;
struct MoeArgs {
  const void* x;
  int64_t ldx;
  const void* router;
  int64_t ldr;
  const uint8_t *up, *up_scales;
  int64_t ldu;
  const uint8_t *down, *down_scales;
  int64_t ldd;
  void* y;
  int64_t ldy;
  int32_t* experts;
  float* weights;
  int64_t T, E, top, H, I;
};
// Bytes of workspace, and where its five parts start.
size_t moe_workspace(const MoeArgs& a, size_t (&at)[5]);
cudaError_t launch_moe(const MoeArgs& a, void* workspace, uint32_t* control, const DeviceCtl& ctl,
                       cudaStream_t s);

}  // namespace mx
}  // namespace mhr
