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

cudaError_t launch_sort(const int32_t* experts, int64_t n, int64_t E, int32_t* offsets,
                        int32_t* order, cudaStream_t s);

}  // namespace routed
}  // namespace mhr
