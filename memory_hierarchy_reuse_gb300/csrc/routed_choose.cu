// The router: which experts a token goes to, with what weights, and the gradient
// of the logits (gemm_routed_choose, gemm_routed_choose_grad).
//
// A warp takes a token.  Its lanes split into `groups` runs of `per` lanes (a power
// of two), a run holds one group's logits in registers, neighbours in neighbouring
// registers; so a group's two best are a few shuffles inside the run, and the first
// lane and register with a value is the one of the lowest index.  Each lane sorts its
// keys; the best of all are then taken one by one from the lists' heads.
//
// Bound by the issue of instructions, not by the logits' bytes (16384 x 256 fp32 logits
// are 2.5 us of the memory's time and take 21 us on a GB300, 1005 instructions a token; one
// token 4.4 us call after call, its gradient as much): keys are integers that order as the floats do,
// sorted by minima and maxima alone, their indices found again for the chosen; a token
// with a NaN, or with keys too near for 32 bits, is done again in double by a function
// of its own.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "mhr_mxfp4.h"
#include "mhr_routed.h"
#include "mxfp4_common.cuh"
#include "routed_internal.h"

namespace mhr {
namespace routed {
namespace {

using mx::from_float;
using mx::to_float;

constexpr uint32_t ALL = 0xffffffffu;
constexpr int WARPS = 4;  // tokens a block

__device__ __forceinline__ float infinity() { return __int_as_float(0x7f800000); }

// Keys as unsigned numbers in the same order: -0 and 0 are one, every NaN is the
// largest, and 0 (below -inf) stands for what cannot be chosen.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return v != v ? ALL : b ^ (b >> 31 ? ALL : 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return v != v ? ~0ull : b ^ (b >> 63 ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return k == ALL ? __uint_as_float(0x7fffffffu)
                  : __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ double key_value(uint64_t k) {
  return k == ~0ull ? __longlong_as_double(0x7fffffffffffffffll)
                    : __longlong_as_double(static_cast<long long>(k >> 63 ? k ^ (1ull << 63) : ~k));
}

__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(ALL, static_cast<uint32_t>(k >> 32));
  const uint32_t lo =
      __reduce_max_sync(ALL, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
  return static_cast<uint64_t>(hi) << 32 | lo;
}

__device__ __forceinline__ float warp_max_float(float v) {
  return key_value(__reduce_max_sync(ALL, ordered(v)));
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(ALL, v, m);
  return v;
}

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
__device__ __forceinline__ float quotient(float a, float b) { return __fdividef(a, b); }  // (2 ulp)
__device__ __forceinline__ double quotient(double a, double b) { return a / b; }
// e^x / (1 + e^x) from the side on which nothing overflows.
template <typename F>
__device__ __forceinline__ F sigmoid(F x) {
  const F e = exp_of(x < 0 ? x : -x);
  return quotient(x < 0 ? e : F(1), 1 + e);
}

struct ChooseParams {
  const void* logits;
  const float* bias;
  int32_t* experts;
  float* weights;
  int64_t ld;
  int32_t T, E, top, groups, group_top;
  int32_t size, per, each;  // experts a group, lanes a group (2^per_log2), experts a lane
  int32_t per_log2;
  int32_t score, top2, renormalize, vec;
  int32_t vec_bias;
  float scale;
};

// V logits of a lane from `at` on; those past `left` are -inf.
template <typename T, int V>
__device__ __forceinline__ void load_lane(const T* at, int left, bool vec, float (&l)[V]) {
  constexpr int BYTES = V * sizeof(T) < 16 ? V * sizeof(T) : 16, N = BYTES / sizeof(T);
  if (vec && left >= V) {
    using Word = std::conditional_t<BYTES == 16, uint4,
                                    std::conditional_t<BYTES == 8, uint2,
                                    std::conditional_t<BYTES == 4, uint32_t, uint16_t>>>;
#pragma unroll
    for (int i = 0; i < V; i += N) {
      const Word w = *reinterpret_cast<const Word*>(at + i);
      T e[N];
      memcpy(e, &w, sizeof(w));
#pragma unroll
      for (int j = 0; j < N; ++j) l[i + j] = to_float(e[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = i < left ? to_float(at[i]) : -infinity();
  }
}

// Of a softmax: the row's maximum and its sum; 0 for both where all are -inf.
template <typename F, int V>
__device__ __forceinline__ void softmax_sums(const float (&l)[V], int count, float& most, F& sum) {
  most = -infinity();
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < count) most = key_value(max(ordered(most), ordered(l[i])));
  most = warp_max_float(most);
  F part = 0;
  if (most > -infinity() || most != most) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < count) part += exp_of(static_cast<F>(l[i]) - static_cast<F>(most));
  }
  sum = warp_sum(part);
  if (sum == 0) most = 0;
}

template <typename F>
__device__ __forceinline__ F score_of(float l, int kind, float most, F sum) {
  if (kind == MHR_SIGMOID) return sigmoid(static_cast<F>(l));
  return sum == 0 ? F(0) : exp_of(static_cast<F>(l) - static_cast<F>(most)) / sum;
}

// The lanes' share of the row: group, first expert, number of experts.
struct Share {
  int group, first, count;
};
__device__ __forceinline__ Share share_of(const ChooseParams& p, int lane) {
  Share s;
  s.group = lane >> p.per_log2;
  const int sub = lane & (p.per - 1);
  s.count = s.group < p.groups ? max(0, min(p.each, p.size - sub * p.each)) : 0;
  s.first = s.count ? s.group * p.size + sub * p.each : 0;
  return s;
}

// The choice in double: lane j <= top gets the j-th best expert (-1 past the last) and
// its logit; most and sum are the softmax's.  Every NaN is the largest.
struct Choice {
  int expert;
  float logit, most, sum;
};
// Few tokens come here, one or two at a time, so it is short, in loops over the shared
// memory at `work` (32 V numbers): unrolled, 14 us of such a token's time went by until
// its instructions were there.
template <typename T, int V>
__device__ __noinline__ Choice choose_double(const ChooseParams& p, int t, int lane,
                                             uint64_t* work) {
  const Share sh = share_of(p, lane);
  const T* row = static_cast<const T*>(p.logits) + t * p.ld + sh.first;
  const bool scored = p.bias != nullptr, softmax = p.score == MHR_SOFTMAX;
  const bool sums = p.groups > 1 && p.top2;
  uint32_t high = 0;  // (ordered: below -inf)
#pragma unroll 1
  for (int i = 0; i < sh.count; ++i) high = max(high, ordered(to_float(row[i])));
  float most = key_value(__reduce_max_sync(ALL, high));
  if (most == -infinity()) most = 0;
  uint64_t* mine = work + lane;  // every 32nd
  double part = 0;
#pragma unroll 1
  for (int i = 0; i < sh.count; ++i) {
    const double x = to_float(row[i]);
    const double e = exp(softmax ? x - most : -fabs(x));
    mine[32 * i] = __double_as_longlong(e);
    part += e;
  }
  const double sum = softmax ? warp_sum(part) : 0;
  uint64_t score1 = 0, score2 = 0;  // the lane's two best scores, where groups add up scores
  uint64_t best = 0;                // and its best key
#pragma unroll 1
  for (int i = 0; i < sh.count; ++i) {
    const double x = to_float(row[i]), e = __longlong_as_double(mine[32 * i]);
    const double of = softmax ? (sum == 0 ? 1.0 : sum) : 1 + e;
    const double s = (!softmax && x >= 0 ? 1.0 : e) / of + (scored ? p.bias[sh.first + i] : 0.f);
    const uint64_t k = ordered(s), key = scored ? k : ordered(x);
    score2 = max(score2, min(score1, k));
    score1 = max(score1, k);
    best = max(best, key);
    mine[32 * i] = key;
  }
  if (p.groups > 1) {
    uint64_t worth = best;
    if (sums) worth = score1;
    for (int m = 1; m < p.per; m <<= 1) {
      const uint64_t o1 = __shfl_xor_sync(ALL, worth, m), o2 = __shfl_xor_sync(ALL, score2, m);
      score2 = max(max(score2, o2), min(worth, o1));
      worth = max(worth, o1);
    }
    // (a group of one has no second)
    if (sums && worth && p.size > 1) worth = ordered(key_value(worth) + key_value(score2));
    bool open = false;
#pragma unroll 1
    for (int g = 0; g < p.group_top; ++g) {
      const uint64_t m = warp_max(open ? uint64_t{0} : worth);
      if (sh.group == (__ffs(__ballot_sync(ALL, !open && worth == m)) - 1) >> p.per_log2)
        open = true;
    }
    if (!open) best = 0;
  }
  Choice c{-1, 0.f, most, static_cast<float>(sum)};
#pragma unroll 1
  for (int j = 0; j <= p.top; ++j) {
    const uint64_t m = warp_max(best);
    if (m == 0) break;
    const int owner = __ffs(__ballot_sync(ALL, best == m)) - 1;
    int at = 0;
    if (lane == owner) {  // takes the first of it, and looks for its next
      while (at + 1 < sh.count && mine[32 * at] != m) ++at;
      mine[32 * at] = 0;
      best = 0;
#pragma unroll 1
      for (int i = 0; i < sh.count; ++i) best = max(best, mine[32 * i]);
    }
    const int e = __shfl_sync(ALL, sh.first + at, owner);
    if (lane == j) c.expert = e;
  }
  if (c.expert >= 0) c.logit = to_float(row[c.expert - sh.first]);
  return c;
}

// Floats that are no NaN as signed integers in the same order; -0 has to be 0.
__device__ __forceinline__ int sortable(float v) {
  const int b = __float_as_int(v);
  return b ^ (b >> 31 & 0x7fffffff);
}
__device__ __forceinline__ float of_sortable(int k) {
  return __int_as_float(k ^ (k >> 31 & 0x7fffffff));
}
constexpr int NONE = -0x7fffffff - 1;  // below every key

// Descending, by a merge-exchange network.
template <int V>
__device__ __forceinline__ void sort_descending(int (&k)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const int a = k[i + j], b = k[i + j + q];
            k[i + j] = max(a, b);
            k[i + j + q] = min(a, b);
          }
}

// How far two keys may be off together.  A sigmoid's score: expf's 2 ulp, a sum and a
// quotient of 2 ulp, 5 * 2^-23 of it at most.  A softmax's, in parts of 2^-24: 4 of expf, 4
// and 1 of the quotient and the product; 40 of the sum (36 roundings and its terms'), which
// two scores share, so that the difference is off by half of that for each; and its rounded
// argument, at most ln(1 / score): 7 down to 2^-10, 88 down to 2^-126.  Below, all these are
// steps of 2^-149.  The sum with the bias is off by 2^-24 of the key.
__device__ __forceinline__ float near_by(int kind, float s, float s1, float key) {
  const float sum = 0x1p-22f * fabsf(key) + 0x1p-146f;
  if (kind == MHR_SIGMOID) return 0x1p-20f * (s + s1) + sum;
  return 0x1.2p-19f * (s + s1) + 81 * 0x1p-24f * (fminf(s, 0x1p-10f) + fminf(s1, 0x1p-10f)) + sum;
}

// Whether 32 bits do not tell one of this lane's keys from the given one, except for the
// same numbers.
template <typename T, int V>
__device__ __noinline__ bool others_near(const ChooseParams& p, int t, int lane, float logit,
                                         float bias, float key, float s, float most, float sum) {
  const Share sh = share_of(p, lane);
  const T* row = static_cast<const T*>(p.logits) + t * p.ld + sh.first;
  bool near = false;
#pragma unroll 1
  for (int i = 0; i < sh.count; ++i) {
    const float x = to_float(row[i]), b = p.bias[sh.first + i];
    const float s1 = score_of<float>(x, p.score, most, sum);
    near |= !(x == logit && b == bias) &&
            !(fabsf(key - (s1 + b)) > near_by(p.score, s, s1, key));
  }
  return near;
}

// The order of 32 candidates, a lane each, best first but for neighbours too near: by
// their keys in double, neighbour by neighbour until none changes places.
template <typename T, int V>
__device__ __noinline__ Choice refine(const ChooseParams& p, int t, int lane, int expert,
                                      float logit, float most) {
  double sum = 0;
  if (p.score == MHR_SOFTMAX) {
    const Share sh = share_of(p, lane);
    float l[V];
    load_lane<T, V>(static_cast<const T*>(p.logits) + t * p.ld + sh.first, sh.count, p.vec != 0, l);
    double part = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) part += exp(static_cast<double>(l[i]) - most);
    sum = warp_sum(part);
  }
  uint64_t key = 0;
  if (expert >= 0)
    key = ordered(score_of<double>(logit, p.score, most, sum) + p.bias[expert]);
  for (int round = 0, still = 0; round < 32 && still < 2; ++round) {
    const int with = (lane ^ 1) - (round & 1 ? ((lane & 1) ? -2 : 2) : 0);  // the neighbour
    const bool pair = with >= 0 && with < 32;
    const int from = pair ? with : lane;
    const uint64_t k = __shfl_sync(ALL, key, from);
    const int e = __shfl_sync(ALL, expert, from);
    const float x = __shfl_sync(ALL, logit, from);
    // the lower lane takes the better: of equal keys the lower expert; none is the worst
    const bool other_better = k > key || (k == key && k != 0 && e < expert);
    const bool mine_better = key > k || (k == key && k != 0 && expert < e);
    const bool change = pair && (lane < with ? other_better : mine_better);
    if (change) {
      key = k;
      expert = e;
      logit = x;
    }
    still = __any_sync(ALL, change) ? 0 : still + 1;
  }
  return Choice{expert, logit, most, static_cast<float>(sum)};
}

// Whether this lane's group stays, its worth taken in double from the lanes' two best keys:
// the `at0`-th and `at1`-th of their experts (-1: there is none).
template <typename T, int V>
__device__ __noinline__ bool open_in_double(const ChooseParams& p, int t, int lane, int at0,
                                            int at1, float most) {
  const Share sh = share_of(p, lane);
  const T* row = static_cast<const T*>(p.logits) + t * p.ld + sh.first;
  double sum = 0;
  if (p.score == MHR_SOFTMAX) {
#pragma unroll 1
    for (int i = 0; i < sh.count; ++i) sum += exp(static_cast<double>(to_float(row[i])) - most);
    sum = warp_sum(sum);
  }
  uint64_t key[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = i ? at1 : at0;
    key[i] = 0;
    if (at >= 0)
      key[i] = ordered(score_of<double>(to_float(row[at]), p.score, most, sum) +
                       (p.bias ? p.bias[sh.first + at] : 0.f));
  }
  uint64_t score1 = max(key[0], key[1]), score2 = min(key[0], key[1]);
  for (int m = 1; m < p.per; m <<= 1) {
    const uint64_t o1 = __shfl_xor_sync(ALL, score1, m), o2 = __shfl_xor_sync(ALL, score2, m);
    score2 = max(max(score2, o2), min(score1, o1));
    score1 = max(score1, o1);
  }
  if (p.top2 && score1 && p.size > 1) score1 = ordered(key_value(score1) + key_value(score2));
  int rank = 0;
#pragma unroll 1
  for (int g = 0; g < p.groups; ++g) {
    const uint64_t other = __shfl_sync(ALL, score1, g << p.per_log2);
    rank += other > score1 || (other == score1 && g < sh.group);
  }
  return sh.group < p.groups && rank < p.group_top;
}

template <typename T, int V>
__global__ void __launch_bounds__(WARPS * 32) choose_kernel(const __grid_constant__ ChooseParams p) {
  __shared__ alignas(16) int shared[WARPS][2][V * 32];  // keys as they lie, and sorted
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * WARPS + warp;
  if (t >= p.T) return;
  const Share sh = share_of(p, lane);
  grid_dependency_wait();
  float l[V];
  load_lane<T, V>(static_cast<const T*>(p.logits) + t * p.ld + sh.first, sh.count, p.vec != 0, l);

  // Without a bias the logits' own order is the scores'.
  const bool scored = p.bias != nullptr, sums = p.groups > 1 && p.top2;
  const bool softmax = p.score == MHR_SOFTMAX;
  bool again = false;  // in double
  float most = 0, sum = 0;
  if (softmax && (scored || sums || !p.renormalize)) {
    most = -infinity();
#pragma unroll
    for (int i = 0; i < V; ++i) most = fmaxf(most, l[i]);  // (-inf past the count)
    most = of_sortable(__reduce_max_sync(ALL, sortable(most)));
    float part = 0;
    if (most > -infinity()) {
#pragma unroll
      for (int i = 0; i < V; ++i) part += expf(l[i] - most);
    }
    sum = warp_sum(part);
    if (sum == 0) most = 0;
    again = sum != sum;  // (a NaN or an infinity)
  }
  int key[V];
  {
    const float r = sum == 0 ? 0.f : __fdividef(1.f, sum);
    float bias[V];
    if (scored) load_lane<float, V>(p.bias + sh.first, sh.count, p.vec_bias != 0, bias);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float v = l[i] + 0.f;
      if (scored) v = (softmax ? expf(l[i] - most) * r : sigmoid(l[i])) + bias[i];
      if (i >= sh.count) v = 0.f;
      again |= v != v;
      key[i] = i < sh.count ? sortable(v) : NONE;
    }
  }
  const int* originals = shared[warp][0];
  int* original = shared[warp][0] + lane * V;
  int* list = shared[warp][1] + lane * V;
#pragma unroll
  for (int i = 0; i < V; ++i) original[i] = key[i];
  sort_descending<V>(key);
#pragma unroll
  for (int i = 0; i < V; ++i) list[i] = key[i];
  int head = key[0];
  if (p.groups > 1) {
    int best = key[0], second = V > 1 ? key[V > 1 ? 1 : 0] : NONE;
    for (int m = 1; m < p.per; m <<= 1) {
      const int o = __shfl_xor_sync(ALL, best, m);
      if (sums) second = max(max(second, __shfl_xor_sync(ALL, second, m)), min(best, o));
      best = max(best, o);
    }
    int worth = best;
    if (sums && best != NONE) {
      float a = of_sortable(best), b = of_sortable(second);
      if (!scored) {
        a = score_of<float>(a, p.score, most, sum);
        b = score_of<float>(b, p.score, most, sum);
      }
      a = p.size > 1 ? a + b : a;  // (a group of one has no second)
      again |= a != a;
      worth = sortable(a + 0.f);
    }
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const int other = __shfl_sync(ALL, worth, g * p.per);
      rank += other > worth || (other == worth && g < sh.group);
    }
    bool open = sh.group < p.groups && rank < p.group_top;
    if (scored || sums) {  // is the best of the closed ones as good?
      const float a = of_sortable(__reduce_min_sync(ALL, open ? worth : 0x7f800000));
      const int closed = __reduce_max_sync(ALL, open ? NONE : worth);
      // (scores of at most 1: one, or two, of either)
      const float n = sums ? 2.f : 1.f;
      if (closed != NONE && !(a - of_sortable(closed) > near_by(p.score, n, n, 4.f * (fabsf(a) + n)))) {
        // The lanes' best two in double, if the third is not one of them as well.
        const int first = key[0], next = key[V > 1 ? 1 : 0];
        int at0 = -1, at1 = -1;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
          if (i < sh.count && original[i] == first) at0 = i;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
          if (i < sh.count && i != at0 && original[i] == next) at1 = i;
        if (V > 2 && sh.count > 2) {
          const float third = of_sortable(key[V > 2 ? 2 : 0]), second = of_sortable(next);
          again |= !(second - third > near_by(p.score, 1.f, 1.f, 4.f * (fabsf(second) + 1.f)));
        }
        open = open_in_double<T, V>(p, t, lane, at0, at1, most);
      }
    }
    if (!open) head = NONE;
  }
  __syncwarp();
  // The best of the heads, one by one: lane j keeps the j-th, whose it is, and how many
  // equal ones of that lane came before it.
  int mine = NONE, owner = 0, taken = 0;
  auto take = [&](int from, int to) {
    for (int j = from; j < to; ++j) {
      const int m = __reduce_max_sync(ALL, head);
      const int o = __ffs(__ballot_sync(ALL, head == m)) - 1;
      if (lane == j) {
        mine = m;
        owner = o;
      }
      if (lane == o) {
        ++taken;
        head = taken < V && m != NONE ? list[taken] : NONE;
      }
    }
  };
  const T* row = static_cast<const T*>(p.logits) + t * p.ld;
  int expert;
  float logit, s;
  auto look_up = [&](int lanes) {
    const int k1 = __shfl_up_sync(ALL, mine, 1), o1 = __shfl_up_sync(ALL, owner, 1);
    const uint32_t starts = __ballot_sync(ALL, lane == 0 || k1 != mine || o1 != owner);
    int before = lane - (31 - __clz(starts & (0xffffffffu >> (31 - lane))));
    expert = -1;
    if (lane < lanes && mine != NONE) {
      int at = 0;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) at = originals[owner * V + i] == mine ? i : at;
      if (before)  // (equal keys in one lane)
        for (int i = at + 1; i < V && before; ++i)
          if (originals[owner * V + i] == mine) {
            at = i;
            --before;
          }
      expert = (owner >> p.per_log2) * p.size + (owner & (p.per - 1)) * p.each + at;
    }
    logit = expert >= 0 ? to_float(row[expert]) : 0.f;
    s = score_of<float>(logit, p.score, most, sum);
  };
  take(0, p.top + 1);
  look_up(p.top + 1);

  // Neighbours that 32 bits do not tell apart, unless they are the same numbers.  Behind the
  // first key that is not chosen may follow others whose scores, and errors, are larger: the
  // last chosen one is held against the largest score there is (or, where the one behind it
  // is the same, against all).
  const float high_score = softmax && sum > 0.f ? __fdividef(1.f, sum) : 1.f;
  bool near = false;
  if (scored) {
    const float key = of_sortable(mine), key1 = __shfl_down_sync(ALL, key, 1);
    const float l1 = __shfl_down_sync(ALL, logit, 1), s1 = __shfl_down_sync(ALL, s, 1);
    const float b = expert >= 0 ? p.bias[expert] : 0.f, b1 = __shfl_down_sync(ALL, b, 1);
    const int e1 = __shfl_down_sync(ALL, expert, 1);
    const bool equal = logit == l1 && b == b1, last = lane == p.top - 1;
    if (lane < p.top && e1 >= 0)
      near = !equal && !(key - key1 > near_by(p.score, s, last ? high_score : s1, key));
    if (__any_sync(ALL, last && e1 >= 0 && equal)) {
      const int from = p.top - 1;
      near |= others_near<T, V>(p, t, lane, __shfl_sync(ALL, logit, from),
                                __shfl_sync(ALL, b, from), __shfl_sync(ALL, key, from),
                                __shfl_sync(ALL, s, from), most, sum);
    }
  }
  near = __any_sync(ALL, near);
  again = __any_sync(ALL, again);
  if (near && !again) {
    // 32 candidates, if the last of them is out of the question for sure.
    take(p.top + 1, 32);
    look_up(32);
    const float key = of_sortable(mine);
    const float last = __shfl_sync(ALL, key, p.top - 1), s0 = __shfl_sync(ALL, s, p.top - 1);
    const bool far = mine == NONE ||
                     last - key > near_by(p.score, s0, high_score, fabsf(last) + fabsf(key));
    again = !__shfl_sync(ALL, static_cast<int>(far), 31);
  }
  if (again || near) {
    __syncwarp();
    const Choice c = again ? choose_double<T, V>(p, t, lane,
                                                 reinterpret_cast<uint64_t*>(shared[warp][0]))
                           : refine<T, V>(p, t, lane, expert, logit, most);
    expert = c.expert;
    logit = c.logit;
    most = c.most;
    sum = c.sum;
    s = score_of<float>(logit, p.score, most, sum);
  }

  float w = expert >= 0 ? s : 0.f;
  if (p.renormalize) {
    const bool in = lane < p.top;
    const float high = warp_max_float(in ? logit : -infinity());
    // sigmoids of logits this low are e^x but for 1e-26 of them
    if (softmax || high < -60.f) {
      w = in && high != -infinity() ? expf(logit - high) : 0.f;
    } else {
      w = in ? s : 0.f;
    }
    const float total = warp_sum(w);
    w = total == 0 ? 0.f : __fdividef(w, total);
  }
  if (lane < p.top) {
    const int64_t at = static_cast<int64_t>(t) * p.top + lane;
    p.experts[at] = expert;
    p.weights[at] = p.scale * w;
  }
}

// ------------------------------------------------------------------ gradient

struct GradParams {
  const void* logits;
  const int32_t* experts;
  const float* grad;
  void* out;
  int64_t ld, ldg;
  int32_t T, E, top;
  int32_t score, renormalize, vec, vec_out;
  float scale;
};

// A warp takes a token: lane j its j-th expert, every lane V neighbouring columns of
// the row, which the chosen ones' gradients reach through shared memory.
template <typename T, int V>
__global__ void __launch_bounds__(WARPS * 32) choose_grad_kernel(const GradParams p) {
  __shared__ alignas(16) float rows[WARPS][V * 32];
  const int lane = threadIdx.x & 31;
  float* row = rows[threadIdx.x >> 5];
  const int t = blockIdx.x * WARPS + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const T* logits = static_cast<const T*>(p.logits) + t * p.ld;
  const int first = lane * V, count = max(0, min(V, p.E - first));
  const bool whole = p.score == MHR_SOFTMAX && !p.renormalize;

  grid_dependency_wait();
  int e = -1;
  float g = 0, l = -infinity();
  if (lane < p.top) {
    const int64_t at = static_cast<int64_t>(t) * p.top + lane;
    e = p.experts[at];
    g = p.grad[at];
    if (e < 0 || e >= p.E) e = -1;
    if (e >= 0) l = to_float(logits[e]);
  }
  float base[V];
#pragma unroll
  for (int i = 0; i < V; ++i) base[i] = 0;
  float d = 0;  // of this lane's expert
  const bool in = e >= 0;
  if (whole) {
    float x[V], most, sum;
    load_lane<T, V>(logits + (count ? first : 0), count, p.vec != 0, x);
    softmax_sums<float>(x, count, most, sum);
    const float s = in ? score_of<float>(l, MHR_SOFTMAX, most, sum) : 0.f;
    const float dot = warp_sum(in ? s * g : 0.f);
    const float r = sum == 0 ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < count) base[i] = sum == 0 ? 0.f : -p.scale * dot * (expf(x[i] - most) * r);
    d = in ? p.scale * s * g : 0.f;
  } else if (p.renormalize) {
    const float high = warp_max_float(in ? l : -infinity());
    const bool as_softmax = p.score == MHR_SOFTMAX || high < -60.f;
    const float s = p.score == MHR_SIGMOID && in ? sigmoid(l) : 0.f;
    float w = 0;
    if (as_softmax)
      w = in && high != -infinity() ? expf(l - high) : 0.f;
    else
      w = s;
    const float total = warp_sum(w);
    w = total == 0 ? 0.f : w / total;
    const float dot = warp_sum(in ? w * g : 0.f);
    // (1 - s is 1 / (1 + e^l): not lost where s is next to 1)
    const float slope = p.score == MHR_SIGMOID && in ? sigmoid(-l) : 1.f;
    d = in ? p.scale * w * slope * (g - dot) : 0.f;
  } else {
    d = in ? p.scale * g * sigmoid(l) * sigmoid(-l) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) row[first + i] = base[i];
  __syncwarp();
  // One expert twice in a row: its first lane adds all of them up.
  const uint32_t same = __match_any_sync(ALL, in ? e : -1 - lane);
  if (__any_sync(ALL, (same & (same - 1)) != 0)) {
    float total = 0;
    for (int j = 0; j < p.top; ++j) {
      const float dj = __shfl_sync(ALL, d, j);
      if (same >> j & 1) total += dj;
    }
    d = total;
  }
  if (in && __ffs(same) - 1 == lane) row[e] += d;
  __syncwarp();
  T* out = static_cast<T*>(p.out) + t * p.ldg;
  constexpr int N = 16 / sizeof(T);
  if (p.vec_out) {  // 16 bytes a lane, neighbours next to one another
    for (int c = lane * N; c + N <= p.E; c += 32 * N) {
      T v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = from_float<T>(row[c + i]);
      uint4 w;
      memcpy(&w, v, sizeof(w));
      *reinterpret_cast<uint4*>(out + c) = w;
    }
    for (int c = p.E / N * N + lane; c < p.E; c += 32) out[c] = from_float<T>(row[c]);
  } else {
    for (int c = lane; c < p.E; c += 32) out[c] = from_float<T>(row[c]);
  }
}

bool aligned16(const void* p, int64_t pitch_bytes) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && pitch_bytes % 16 == 0;
}
int size_of(int dtype) { return dtype == MHR_F32 ? 4 : 2; }

// f(type tag, values a lane) for the smallest V that holds `each`.
template <typename F>
cudaError_t by_type_and_width(int dtype, int each, const F& f) {
  auto width = [&](auto tag) {
    if (each <= 1) return f(tag, std::integral_constant<int, 1>{});
    if (each <= 2) return f(tag, std::integral_constant<int, 2>{});
    if (each <= 4) return f(tag, std::integral_constant<int, 4>{});
    if (each <= 8) return f(tag, std::integral_constant<int, 8>{});
    if (each <= 16) return f(tag, std::integral_constant<int, 16>{});
    return f(tag, std::integral_constant<int, 32>{});
  };
  if (dtype == MHR_F32) return width(float{});
  if (dtype == MHR_BF16) return width(__nv_bfloat16{});
  return width(__half{});
}

// A warp a token, set up while the kernel before still runs.
template <typename P>
cudaError_t launch_tokens(void (*kern)(P), const P& p, int64_t T, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((T + WARPS - 1) / WARPS));
  cfg.blockDim = dim3(WARPS * 32);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_launch();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_choose(const ChooseArgs& a, cudaStream_t s) {
  ChooseParams p;
  p.logits = a.logits;
  p.bias = a.bias;
  p.experts = a.experts;
  p.weights = a.weights;
  p.ld = a.ld;
  p.T = static_cast<int32_t>(a.T);
  p.E = static_cast<int32_t>(a.E);
  p.top = static_cast<int32_t>(a.top);
  p.groups = a.group_top == a.groups ? 1 : static_cast<int32_t>(a.groups);  // all stay: no choice
  p.group_top = static_cast<int32_t>(a.group_top);
  p.size = p.E / p.groups;
  p.per_log2 = 5;
  while (p.groups << p.per_log2 > 32) --p.per_log2;
  p.per = 1 << p.per_log2;
  p.each = (p.size + p.per - 1) / p.per;
  p.score = a.score;
  p.top2 = a.group_score == MHR_GROUP_TOP2;
  p.renormalize = a.renormalize;
  p.scale = a.scale;
  return by_type_and_width(a.dtype, p.each, [&](auto tag, auto width) {
    constexpr int V = decltype(width)::value;
    // lanes take whole vectors where a group splits into them
    if (p.size % V == 0 && p.size / V <= p.per) p.each = V;
    p.vec = aligned16(a.logits, a.ld * size_of(a.dtype)) && p.each == V && p.size % V == 0;
    p.vec_bias = aligned16(a.bias, 0) && p.each == V && p.size % V == 0;
    return launch_tokens(choose_kernel<decltype(tag), V>, p, a.T, s);
  });
}

cudaError_t launch_choose_grad(const ChooseGradArgs& a, cudaStream_t s) {
  GradParams p;
  p.logits = a.logits;
  p.experts = a.experts;
  p.grad = a.grad_weights;
  p.out = a.grad_logits;
  p.ld = a.ld;
  p.ldg = a.ldg;
  p.T = static_cast<int32_t>(a.T);
  p.E = static_cast<int32_t>(a.E);
  p.top = static_cast<int32_t>(a.top);
  p.score = a.score;
  p.renormalize = a.renormalize;
  p.scale = a.scale;
  p.vec = aligned16(a.logits, a.ld * size_of(a.dtype));
  p.vec_out = aligned16(a.grad_logits, a.ldg * size_of(a.dtype));
  return by_type_and_width(a.dtype, (p.E + 31) / 32, [&](auto tag, auto width) {
    constexpr int V = decltype(width)::value;
    return launch_tokens(choose_grad_kernel<decltype(tag), V>, p, a.T, s);
  });
}

}  // namespace routed
}  // namespace mhr
