// Launchers of the operators that go by an index per row, shared between their
// C-ABI front end (routed_api.cu) and their kernels.  As in mhr_internal.h,
// launchers assume validated arguments (sizes >= 1, pointers non-null) and
// return the launch's cudaError_t.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "mhr_internal.h"

namespace mhr {
namespace routed {

constexpr int64_t MAX_EXPERTS = 512, MAX_TOP = 16, MAX_GROUPS = 32;  // of a router
constexpr int64_t MAX_PARTS = 1024;                                 // of a sort, and its products
constexpr int64_t MAX_RANK = 128;                                   // of an adapter

struct ChooseArgs {
  int dtype;
  const void* logits;
  int64_t T, E, ld;
  int score;
  const float* bias;
  int64_t groups, group_top;
  int group_score;
  int64_t top;
  bool renormalize;
  float scale;
  int32_t* experts;
  float* weights;
};
cudaError_t launch_choose(const ChooseArgs& a, cudaStream_t s);

struct ChooseGradArgs {
  int dtype;
  const void* logits;
  int64_t ld;
  const int32_t* experts;
  const float* grad_weights;
  int64_t T, E, top;
  int score;
  bool renormalize;
  float scale;
  void* grad_logits;
  int64_t ldg;
};
cudaError_t launch_choose_grad(const ChooseGradArgs& a, cudaStream_t s);

// Bytes of scratch that `parts` matrices (rows x cols, 16-bit elements, pitch ld,
// `stride` elements apart) take to be read by TMA: 0 for those that it reads as they
// are; -1 where they leave the address space.  picked: rows of the (one) matrix that an
// index picks, which are put in order there; 0 without.
int64_t operand_bytes(const void* p, int64_t parts, int64_t rows, int64_t cols, int64_t ld,
                      int64_t stride, int64_t picked);
// An operand as TMA reads it.
struct Operand {
  const void* p;
  int64_t rows, ld, stride;
};
// The operand itself, or its copy at *scratch, which moves on by operand_bytes.  offsets
// (or null): parts without rows there are left out; index (or null): `picked` entries,
// each over `top` a row, zeros where it is none.
cudaError_t ready(const void* p, int64_t parts, int64_t rows, int64_t cols, int64_t ld,
                  int64_t stride, const int32_t* offsets, const int32_t* index, int64_t top,
                  int64_t picked, char** scratch, cudaStream_t s, Operand* out);
// Up to so many rows a product picks by TMA's gather, without that.  In us from cold L2 (bf16),
// gathered / put in order, by rows:
//     experts, K, N        64           256          512 (666)    1024 (2000)  8000 (4000)
//     128, 4096, 1536      113 / 119    215 / 218    245 / 250    260 / 263    322 / 283
//     16, 4096, 4096       102 / 107    111 / 109    111 / 109    188 / 117    315 / 137
//     8, 1024, 1024        15.4 / 17.2  18.4 / 17.4  20.5 / 17.7  30.7 / 21.1  30.7 / 23.2
// (in brackets: the rows of the last two lines).  The gather pays below some 20 rows an expert;
// the limit by all rows is off by up to 5 us between.
constexpr int64_t FEW_ROWS = 256;

// One gemm_routed_product (product, transposed) or gemm_routed_weight_grad
// (gradient).  K: columns of x; N: the output's columns.  `w` is the weights, or the
// gradient rows (out_rows x N) that `scatter` picks from.
enum class ProductKind { product, transposed, gradient };
struct ProductArgs {
  ProductKind kind;
  int dtype;
  const void* x;
  int64_t x_rows, ldx;
  const int32_t* gather;
  int64_t top;
  const void* w;
  int64_t ldw, stride_w;
  const int32_t* offsets;
  int64_t E;
  int out_dtype;
  void* out;
  int64_t out_rows, ldo, stride_o;
  const int32_t* scatter;
  int64_t rows, K, N;
};
// scratch: operand_bytes of x, then of w.
cudaError_t launch_product(const ProductArgs& a, void* scratch, const DeviceCtl& ctl,
                           cudaStream_t s);

// One gemm_routed_adapters.
struct AdapterArgs {
  int dtype;
  const void* x;
  int64_t ldx;
  const void* down;
  int64_t ldd, stride_d;
  const void* up;
  int64_t ldu, stride_u;
  const int32_t* which;
  const float* scales;
  int64_t L, rank;
  int out_dtype;
  const void* y;
  int64_t ldy;
  void* out;
  int64_t ldo;
  int64_t T, K, N;
};
int64_t adapters_scratch(const AdapterArgs& a);
cudaError_t launch_adapters(const AdapterArgs& a, void* scratch, const DeviceCtl& ctl,
                            cudaStream_t s);

cudaError_t launch_sort(const int32_t* experts, int64_t n, int64_t E, int32_t* offsets,
                        int32_t* order, cudaStream_t s);

}  // namespace routed
}  // namespace mhr
