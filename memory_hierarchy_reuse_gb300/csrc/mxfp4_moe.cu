// A whole mixture-of-experts layer for up to 64 tokens over 4-bit experts, in
// one launch:
//
//   logits = x R^T, the top experts of each token and their softmax weights,
//   h_p = silu(G_e x_t) * (U_e x_t)           for every chosen pair p = (t, e),
//   y_t = sum over p of weight_p D_e h_p.
//
// Bound by HBM: the chosen experts' weights pass once, 17/32 byte each, with a
// few multiply-adds a weight (as many as tokens chose the expert); the
// smallest calls by the latency of the three dependent steps.  So one
// persistent cooperative grid, a CTA an SM, walks routing, the up product and
// the down product with a grid barrier between each.
//
// The product.  Weights are the 16-row side of mma.sync m16n8k16 (f16 inputs,
// fp32 sums), pairs its 8 columns: at this few columns the tensor core idles
// whichever instruction feeds it, and mma.sync takes its operands from the
// registers that the weights are unpacked into.  Each warp walks 16 rows at a
// time, K in steps of 128 columns (four blocks of 32), which it fetches itself
// by cp.async into its own ring in shared memory, several steps ahead and
// across units: no barrier between warps, and the grid barriers pass while the
// next weights are under way.  In a block, lane 4 g + q takes the 8 codes
// 8 q .. 8 q + 7 of rows g and g + 8: the sum over k does not mind an order, so
// they stand for the instruction's own k indices and need no shuffle.  A
// block's two MMAs start from zero and its scale multiplies the fp32 sum.
//
// Columns in f16: x in bf16 (8 significant bits) and h in fp32 are scaled by a
// power of two per token or pair that puts the largest magnitude in [2^12,
// 2^13), so that values down to 2^-26 of the largest keep f16's 11 bits.  x
// stays exact but for values below 2^-29 of its largest.  h is rounded to 11
// bits, an eighth of the final rounding to bf16.
//
// The partial outputs of a pair go to the workspace, and after a third barrier
// a token's pairs are added in their order and rounded: results do not depend
// on the schedule.
#include "mhr_gemm.h"
#include "mhr_mxfp4.h"
#include "mxfp4_common.cuh"

namespace mhr {
namespace mx {
namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int DEPTH = 6;                       // steps of 128 columns in a warp's ring
constexpr int STEP_BYTES = 16 * 64 + 16 * 4;   // 16 rows' codes and scales
constexpr int RING_BYTES = WARPS * DEPTH * STEP_BYTES;
constexpr int MAX_PAIRS = MOE_MAX_TOKENS * MOE_MAX_TOP;
constexpr int MAX_SEGMENTS = 256;
constexpr uint32_t kErrTimeoutGrid = 1u << 4;  // status word: a grid barrier's wait ran out

struct MoeParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* router;
  int64_t ldx, ldr;
  const uint8_t *up, *up_s, *down, *down_s;
  int64_t ldu, ldd;
  __nv_bfloat16* y;
  int64_t ldy;
  int32_t* experts;
  float* weights;
  int32_t T, E, top, H, I;
  int32_t kt_h, kt_i;      // steps of 128 columns along H and I
  // workspace
  float* logits;           // T x E
  float* x_mult;           // T: the power of two that x is scaled by for f16
  uint32_t* h_max;         // T * top: bits of the largest |h| of a pair
  float* h;                // T * top x 128 kt_i
  float* part;             // T * top x H: weight_p D_e h_p
  uint32_t* control;       // [0] barrier arrivals, [1] exits
  int32_t stage_bytes;     // shared memory for staged columns
  uint32_t* status;
  uint64_t wait_limit_ns;
  int32_t inject_stall;
};

// A CTA's part of an expert's units, for some of its pairs.
struct Segment {
  int32_t expert, first, count;   // pairs list[first .. first + count)
  int32_t tile;                   // first unit of the expert
  int32_t item, items;            // place in the CTA's walk, units
  int32_t column;                 // where the pairs' columns are staged
  int32_t run;                    // staged together with the others of its run
};

struct Routing {  // shared memory
  float weight[MAX_PAIRS];
  int16_t expert[MAX_PAIRS];      // of pair t * top + k
  int16_t list[MAX_PAIRS];        // pairs, expert by expert
  int32_t count[MOE_MAX_EXPERTS];    // pairs of an expert
  int16_t offset[MOE_MAX_EXPERTS];   // its first place in list
  int16_t active[MOE_MAX_EXPERTS];   // the experts that some pair has
  Segment seg[MAX_SEGMENTS];
  int32_t num_active, segments, items;
  int32_t last, abort;
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// c = a b, and c += a b.
__device__ __forceinline__ void mma_f16_16x8x16_first(float (&c)[4], uint32_t a0, uint32_t a1,
                                                      uint32_t a2, uint32_t a3, uint32_t b0,
                                                      uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_f16_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1,
                                                uint32_t a2, uint32_t a3, uint32_t b0,
                                                uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four scale codes of a row as floats (code 0 is 2^-127, 255 NaN; exact).
__device__ __forceinline__ void scales4(uint32_t codes, float (&f)[4]) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %0, l;\n\tcvt.rn.bf16x2.ue8m0x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
  f[0] = __uint_as_float(lo << 16);
  f[1] = __uint_as_float(lo & 0xffff0000u);
  f[2] = __uint_as_float(hi << 16);
  f[3] = __uint_as_float(hi & 0xffff0000u);
}

// The power of two that puts a magnitude with these fp32 bits in [2^12, 2^13);
// 1 for zero, infinities and NaNs (which f16 keeps).
__device__ __forceinline__ float f16_multiplier(uint32_t amax) {
  const int e = static_cast<int>(amax >> 23);
  if (amax == 0 || e == 255) return 1.f;
  const int m = 127 + 12 - (e - 127);  // biased exponent of the multiplier
  return __uint_as_float(static_cast<uint32_t>(min(max(m, 1), 254)) << 23);
}

__device__ __forceinline__ uint4 to_f16x8(const float (&v)[8], float mult) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i] * mult, v[2 * i + 1] * mult);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// All CTAs of the (cooperative) grid; bounded.  Returns false when the wait
// ran out or another thread of the CTA had given up.
__device__ bool grid_barrier(const MoeParams& p, Routing& r, uint32_t round) {
  __syncthreads();
  if (threadIdx.x == 0 && !r.abort) {
    __threadfence();
    const bool absent = p.inject_stall && blockIdx.x == 0 && round == 1;  // test hook
    if (!absent) atomicAdd(p.control, 1u);
    const uint32_t want = round * gridDim.x;
    const uint64_t t0 = global_timer_ns();
    volatile uint32_t* arrivals = p.control;
    while (*arrivals < want) {
      if (global_timer_ns() - t0 > p.wait_limit_ns) {
        atomicOr(p.status, kErrTimeoutGrid);
        r.abort = 1;
        break;
      }
    }
    __threadfence();
  }
  __syncthreads();
  return r.abort == 0;
}

// N times 8 columns k, k + 256, ... of a bf16 row (zeros past the end), as
// loaded: all loads are under way before the first is used.
template <int N>
__device__ __forceinline__ void load_row(const __nv_bfloat16* row, int k, int cols, bool vec,
                                         uint4 (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int left = cols - (k + 256 * i);
    if (vec && left >= 8) {
      v[i] = __ldg(reinterpret_cast<const uint4*>(row + k + 256 * i));
    } else {
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(row + k + 256 * i + 2 * j);
        u[j] = (2 * j < left ? h[0] : 0u) | ((2 * j + 1 < left ? h[1] : 0u) << 16);
      }
      v[i] = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
}
__device__ __forceinline__ void unpack_bf16(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// Step 1, all warps of the grid: router logits, a warp one expert and TT tokens.
template <int TT>
__device__ void route_logits(const MoeParams& p, int warp, int warps, bool vx, bool vr) {
  const int lane = threadIdx.x & 31;
  const int sets = (p.T + TT - 1) / TT;
  constexpr int N = TT == 1 ? 8 : 4;  // loads of 8 columns a row in flight
  for (int task = warp; task < p.E * sets; task += warps) {
    const int e = task / sets, t0 = (task - e * sets) * TT;
    float sum[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) sum[j] = 0.f;
    for (int k = lane * 8; k < p.H; k += 256 * N) {
      uint4 w[N], x[TT][N];
      load_row<N>(p.router + e * p.ldr, k, p.H, vr, w);
#pragma unroll
      for (int j = 0; j < TT; ++j) load_row<N>(p.x + min(t0 + j, p.T - 1) * p.ldx, k, p.H, vx, x[j]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float wf[8];
        unpack_bf16(w[i], wf);
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          float xf[8];
          unpack_bf16(x[j][i], xf);
#pragma unroll
          for (int c = 0; c < 8; ++c) sum[j] = fmaf(wf[c], xf[c], sum[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < TT; ++j) {
#pragma unroll
      for (int d = 16; d; d >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], d);
      if (lane == 0 && t0 + j < p.T) p.logits[(t0 + j) * p.E + e] = sum[j];
    }
  }
}

// Step 1 also: each token's f16 multiplier and zeroed maxima of its pairs.
__device__ void route_start(const MoeParams& p) {
  const int lane = threadIdx.x & 31;
  const int warp = (threadIdx.x >> 5) * gridDim.x + blockIdx.x;  // neighbours on other SMs
  const int warps = gridDim.x * WARPS;
  const bool vx = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ldx % 8 == 0;
  const bool vr = reinterpret_cast<uintptr_t>(p.router) % 16 == 0 && p.ldr % 8 == 0;
  for (int t = warps - 1 - warp; t < p.T; t += warps) {  // the warps with fewest logits
    uint32_t amax = 0;
    for (int k = lane * 8; k < p.H; k += 256 * 8) {
      uint4 x[8];
      load_row<8>(p.x + t * p.ldx, k, p.H, vx, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          amax = max(amax, max((u[j] << 16) & 0x7fffffffu, u[j] & 0x7fff0000u));
      }
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if (lane == 0) p.x_mult[t] = f16_multiplier(amax);
    if (lane < p.top) p.h_max[t * p.top + lane] = 0;
  }
  if (p.E * p.T <= warps)
    route_logits<1>(p, warp, warps, vx, vr);
  else
    route_logits<4>(p, warp, warps, vx, vr);
}

// The chosen experts of one token and their weights, by one warp; PER_LANE x 32
// experts at most.  Logits become unsigned keys of the same order (a NaN
// largest, -0 and 0 alike), 0 for one taken or none.
template <int PER_LANE>
__device__ void choose_token(const MoeParams& p, Routing& r, int t) {
  const int lane = threadIdx.x & 31;
  uint32_t key[PER_LANE];
#pragma unroll
  for (int i = 0; i < PER_LANE; ++i) {
    const int e = lane + 32 * i;
    const float v = e < p.E ? __ldcg(p.logits + t * p.E + e) + 0.f : 0.f;
    const uint32_t b = __float_as_uint(v);
    key[i] = e >= p.E ? 0u : v != v ? 0xffffffffu : b >> 31 ? ~b : b | 0x80000000u;
  }
  uint32_t chosen = 0, first = 0;
  for (int k = 0; k < p.top; ++k) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) m = max(m, key[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    uint32_t e = 0xffffffffu;
#pragma unroll
    for (int i = PER_LANE - 1; i >= 0; --i)
      if (key[i] == m) e = lane + 32 * i;
    e = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i)
      if (e == static_cast<uint32_t>(lane + 32 * i)) key[i] = 0;
    if (k == 0) first = m;
    if (lane == k) {
      chosen = m;
      r.expert[t * p.top + k] = static_cast<int16_t>(e);
    }
  }
  auto logit = [](uint32_t key) {
    return __uint_as_float(key == 0xffffffffu ? key : key >> 31 ? key & 0x7fffffffu : ~key);
  };
  const float w = lane < p.top ? expf(logit(chosen) - logit(first)) : 0.f;
  float sum = w;
#pragma unroll
  for (int d = 8; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane < p.top) r.weight[t * p.top + lane] = w / sum;
}

// Step 2, in every CTA alike: the top experts of each token, ties to the lowest
// index, their weights, and the pairs sorted by expert.
__device__ void route_choose(const MoeParams& p, Routing& r) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int t = warp; t < p.T; t += WARPS) {
    if (p.E <= 128)
      choose_token<4>(p, r, t);
    else
      choose_token<MOE_MAX_EXPERTS / 32>(p, r, t);
  }
  const int pairs = p.T * p.top;
  for (int e = threadIdx.x; e < p.E; e += THREADS) r.count[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += THREADS) atomicAdd(&r.count[r.expert[i]], 1);
  __syncthreads();
  if (warp == 0) {
    int active = 0, offset = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int c = e0 + lane < p.E ? r.count[e0 + lane] : 0;
      const uint32_t has = __ballot_sync(0xffffffffu, c > 0);
      int scan = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += o;
      }
      if (e0 + lane < p.E) r.offset[e0 + lane] = static_cast<int16_t>(offset + scan - c);
      if (c > 0)
        r.active[active + __popc(has & ((1u << lane) - 1))] = static_cast<int16_t>(e0 + lane);
      active += __popc(has);
      offset += __shfl_sync(0xffffffffu, scan, 31);
    }
    if (lane == 0) r.num_active = active;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += THREADS) {
    const int e = r.expert[i];
    // an expert's pairs, from its list's end down, in any order: each is a
    // column of its own (this takes count to zero)
    r.list[r.offset[e] + atomicSub(&r.count[e], 1) - 1] = static_cast<int16_t>(i);
    if (blockIdx.x == 0) {
      p.experts[i] = e;
      p.weights[i] = r.weight[i];
    }
  }
  __syncthreads();
}

// The CTA's equal share of all units (of `tiles` per active expert) as
// segments: expert by expert, at most `most` of an expert's pairs at a time (more
// pairs take its units again), in runs whose columns fit `capacity` together.
__device__ void plan_segments(Routing& r, int pairs, int tiles, int most, int capacity) {
  if (threadIdx.x == 0) {
    // (at most 512 experts x 2048 units x some hundred CTAs: 32 bits)
    const uint32_t units = static_cast<uint32_t>(r.num_active) * tiles;
    const int begin = static_cast<int>(units * blockIdx.x / gridDim.x);
    const int end = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
    int n = 0, item = 0, run = 0, column = 0;
    for (int u = begin; u < end;) {
      const int ai = u / tiles, e = r.active[ai], tile = u - ai * tiles;
      const int items = min(tiles - tile, end - u);
      const int first = r.offset[e];
      const int last = ai + 1 < r.num_active ? r.offset[r.active[ai + 1]] : pairs;
      for (int c = first; c < last && n < MAX_SEGMENTS; c += most) {
        const int count = min(most, last - c);
        if (column + count > capacity) {
          ++run;
          column = 0;
        }
        r.seg[n++] = Segment{e, c, count, tile, item, items, column, run};
        column += count;
        item += items;
      }
      u += items;
    }
    r.segments = n;
    r.items = item;
  }
  __syncthreads();
}

// Steps 3 and 4.  UP: units of 8 gate rows and the same 8 up rows, columns x,
// K = H; otherwise units of 16 rows of the down matrix, columns h, K = I.
// Warps take the CTA's units in turn; of the units left when no full round
// remains, groups of ws warps take one each, every warp an equal part of K.
template <int NT, bool UP>
struct Product {
  const MoeParams& p;
  Routing& r;
  uint8_t* staged;
  uint8_t* ring;       // this warp's
  float* red;          // partial sums of groups: WARPS x NT x 128
  int lane, warp, g, q;
  int kt, blocks, pitch;
  int rounds;                  // the first `rounds` units a whole warp each
  int groups, ws, group, part, k_begin, k_end;  // the others
  // the fetching cursor: unit `item` of the walk, in segment seg, at step lk
  // up to l_end
  int item, seg, lk, l_end, fetched;
  const uint8_t *pa, *pb, *ps;

  __device__ Product(const MoeParams& p_, Routing& r_, uint8_t* staged_, uint8_t* ring0,
                     float* red_)
      : p(p_), r(r_), staged(staged_), red(red_) {
    lane = threadIdx.x & 31;
    warp = threadIdx.x >> 5;
    g = lane >> 2;
    q = lane & 3;
    ring = ring0 + warp * (DEPTH * STEP_BYTES);
    kt = UP ? p.kt_h : p.kt_i;
    blocks = UP ? (p.H + 31) / 32 : (p.I + 31) / 32;
    pitch = kt * 256 + 64;  // 64 past a multiple of 128: neighbouring columns' banks differ
    plan_segments(r, p.T * p.top, UP ? (p.I + 7) / 8 : (p.H + 15) / 16,
                  min(8 * NT, p.stage_bytes / pitch), p.stage_bytes / pitch);
    rounds = r.items & ~(WARPS - 1);
    ws = WARPS;
    while (ws > 2 && (WARPS / ws < r.items - rounds || ws > kt)) ws >>= 1;
    groups = WARPS / ws;
    group = warp / ws;
    part = warp - group * ws;
    k_begin = kt * part / ws;
    k_end = kt * (part + 1) / ws;
    item = rounds ? warp : group;
    seg = 0;
    fetched = 0;
    find();
    for (int d = 0; d < DEPTH - 1; ++d) fetch();
  }

  // The segment and rows of `item`.
  __device__ void find() {
    lk = item < rounds ? 0 : k_begin;
    l_end = item < rounds ? kt : k_end;
    if (item >= r.items || lk == l_end) {
      item = 0x7fffffff;
      return;
    }
    while (item >= r.seg[seg].item + r.seg[seg].items) ++seg;
    const Segment& sg = r.seg[seg];
    const int tile = sg.tile + item - sg.item;
    const int64_t e = sg.expert;
    const uint8_t* data = UP ? p.up : p.down;
    const int64_t ld = UP ? p.ldu : p.ldd;
    auto row_of = [&](int i) {  // row i of the unit's 16; past the last row: the last
      return UP ? (e * 2 + (i >> 3)) * p.I + min(tile * 8 + (i & 7), p.I - 1)
                : e * p.H + min(tile * 16 + i, p.H - 1);
    };
    pa = data + row_of(g) * ld + q * 16;
    pb = data + row_of(g + 8) * ld + q * 16;
    ps = (UP ? p.up_s : p.down_s) + scale_offset(row_of(lane & 15), 0, kt);
  }

  // The warp's unit after `item`.
  __device__ int next(int item) const {
    if (item >= rounds) return item + groups;
    return item + WARPS < rounds ? item + WARPS : rounds + group;
  }

  // One step of 128 columns into the ring (an empty group past the end): row
  // i's block b at place b ^ (i / 2 % 4) of its 64 bytes, so that eight rows'
  // words of a block fall into different banks.
  __device__ void fetch() {
    if (item != 0x7fffffff) {
      const uint32_t st = smem_u32(ring) + fetched * STEP_BYTES;
      const uint32_t at = st + g * 64 + ((q ^ ((g >> 1) & 3)) << 4);
      const uint32_t bytes = lk * 4 + q < blocks ? 16 : 0;  // 0: zero codes
      const int64_t step = bytes ? lk * 64 : 0;
      cp_async_16(at, pa + step, bytes);
      cp_async_16(at + 512, pb + step, bytes);
      if (lane < 16) cp_async_4(st + 1024 + lane * 4, ps + static_cast<int64_t>(lk) * 512);
      if (++fetched == DEPTH) fetched = 0;
      if (++lk == l_end) {
        item = next(item);
        find();
      }
    }
    cp_async_commit();
  }

  // The columns of a run's pairs in f16, in batches of loads.
  __device__ void stage(int run) {
    const int pieces = kt * 16;  // of 8 columns
    const bool vx = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ldx % 8 == 0;
    constexpr int BATCH = UP ? 4 : 2;
    for (int s = 0; s < r.segments; ++s) {
      const Segment sg = r.seg[s];
      if (sg.run != run) continue;
      for (int i0 = threadIdx.x; i0 < sg.count * pieces; i0 += THREADS * BATCH) {
        uint4 raw[BATCH][UP ? 1 : 2];
        float mult[BATCH];
        uint32_t to[BATCH];
        int left[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
          const int i = min(i0 + j * THREADS, sg.count * pieces - 1);  // (past the end: the last)
          const int c = i / pieces, k = (i - c * pieces) * 8, pair = r.list[sg.first + c];
          to[j] = (sg.column + c) * pitch + k * 2;
          if (UP) {
            const int t = pair / p.top;
            mult[j] = __ldcg(p.x_mult + t);
            load_row<1>(p.x + t * p.ldx, k, p.H, vx, *reinterpret_cast<uint4(*)[1]>(raw[j]));
          } else {
            mult[j] = __uint_as_float(__ldcg(p.h_max + pair));
            left[j] = p.I - k;
            const uint4* src = reinterpret_cast<const uint4*>(
                p.h + static_cast<int64_t>(pair) * p.kt_i * 128 + k);
            raw[j][0] = __ldcg(src);
            raw[j][UP ? 0 : 1] = __ldcg(src + 1);
          }
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
          float v[8];
          if (UP) {
            unpack_bf16(raw[j][0], v);
          } else {
            const uint4 a = raw[j][0], b = raw[j][UP ? 0 : 1];
            const uint32_t f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            mult[j] = f16_multiplier(__float_as_uint(mult[j]));
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = c < left[j] ? __uint_as_float(f[c]) : 0.f;
          }
          *reinterpret_cast<uint4*>(staged + to[j]) = to_f16x8(v, mult[j]);
        }
      }
    }
  }

  // Sums of row g (0) or g + 8 (1) of the unit, column n * 8 + 2 q + i.
  __device__ void up_output(const Segment& sg, int tile, int n, int i, float gate, float value) {
    const int col = n * 8 + q * 2 + i, row = tile * 8 + g;
    const bool in = col < sg.count && row < p.I;
    const int pair = r.list[sg.first + min(col, sg.count - 1)];
    const float back = 1.f / __ldcg(p.x_mult + pair / p.top);  // a power of two
    gate *= back;
    value *= back;
    const float h = gate / (1.f + expf(-gate)) * value;
    if (in) p.h[static_cast<int64_t>(pair) * p.kt_i * 128 + row] = h;
    uint32_t m = in ? __float_as_uint(h) & 0x7fffffffu : 0u;
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (g == 0 && col < sg.count) atomicMax(p.h_max + pair, m);
  }
  __device__ void down_output(const Segment& sg, int tile, int n, int i, float v) {
    const int col = n * 8 + q * 2 + (i & 1), row = tile * 16 + g + (i >> 1) * 8;
    if (col < sg.count && row < p.H) {
      const int pair = r.list[sg.first + col];
      const float back = 1.f / f16_multiplier(__ldcg(p.h_max + pair));
      p.part[static_cast<int64_t>(pair) * p.H + row] = v * back * r.weight[pair];
    }
  }

  __device__ void finish(const Segment& sg, int tile, int ntiles, bool whole, float (&acc)[NT][4]) {
    if (whole) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n >= ntiles) break;
        if (UP) {
#pragma unroll
          for (int i = 0; i < 2; ++i) up_output(sg, tile, n, i, acc[n][i], acc[n][2 + i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) down_output(sg, tile, n, i, acc[n][i]);
        }
      }
      return;
    }
    // the group's parts of K, added in their order
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (n < ntiles)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[warp * (NT * 128) + (n * 4 + i) * 32 + lane] = acc[n][i];
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(ws * 32) : "memory");
    const float* mine = red + group * ws * (NT * 128);
    for (int o = part; o < ntiles * (UP ? 2 : 4); o += ws) {
      const int n = UP ? o >> 1 : o >> 2, i = UP ? o & 1 : o & 3;
      float a = 0.f, b = 0.f;
      for (int w = 0; w < ws; ++w) {
        a += mine[w * (NT * 128) + (n * 4 + i) * 32 + lane];
        if (UP) b += mine[w * (NT * 128) + (n * 4 + 2 + i) * 32 + lane];
      }
      if (UP)
        up_output(sg, tile, n, i, a, b);
      else
        down_output(sg, tile, n, i, a);
    }
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(ws * 32) : "memory");
  }

  __device__ void run() {
    int at = 0, run = 0, s = 0;  // ring position; staged run; segment
    if (r.segments) stage(0);
    __syncthreads();
    for (int it = rounds ? warp : group; it < r.items; it = next(it)) {
      const bool whole = it < rounds;
      while (it >= r.seg[s].item + r.seg[s].items) ++s;
      const Segment sg = r.seg[s];
      while (run < sg.run) restage(++run);
      const int ntiles = (sg.count + 7) / 8;
      const uint8_t* column[NT];  // this lane's columns (past the last: the last)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        column[n] = staged + (sg.column + min(n * 8 + g, sg.count - 1)) * pitch + q * 16;
      float acc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
#pragma unroll 1
      for (int k = whole ? 0 : k_begin; k < (whole ? kt : k_end); ++k) {
        cp_async_wait<DEPTH - 2>();
        __syncwarp();  // the step is there for all lanes, and all have read the one before it,
        fetch();       // whose place this takes
        const uint8_t* st = ring + at * STEP_BYTES;
        if (++at == DEPTH) at = 0;
        // everything of the step first, then four blocks with nothing to wait for
        const uint32_t sa = *reinterpret_cast<const uint32_t*>(st + 1024 + g * 4);
        const uint32_t sb = *reinterpret_cast<const uint32_t*>(st + 1024 + g * 4 + 32);
        const uint8_t* row = st + g * 64 + q * 4;
        uint32_t wa[4], wb[4];
        uint4 x[NT][4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          wa[b] = *reinterpret_cast<const uint32_t*>(row + ((b ^ ((g >> 1) & 3)) << 4));
          wb[b] = *reinterpret_cast<const uint32_t*>(row + 512 + ((b ^ ((g >> 1) & 3)) << 4));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (n < ntiles) x[n][b] = *reinterpret_cast<const uint4*>(column[n] + k * 256 + b * 64);
        float fa[4], fb[4];
        scales4(sa, fa);
        scales4(sb, fb);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t a0 = e2m1_to_f16x2<0>(wa[b]), a1 = e2m1_to_f16x2<1>(wa[b]);
          const uint32_t a2 = e2m1_to_f16x2<2>(wa[b]), a3 = e2m1_to_f16x2<3>(wa[b]);
          const uint32_t b0 = e2m1_to_f16x2<0>(wb[b]), b1 = e2m1_to_f16x2<1>(wb[b]);
          const uint32_t b2 = e2m1_to_f16x2<2>(wb[b]), b3 = e2m1_to_f16x2<3>(wb[b]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (n < ntiles) {
              float sum[4];
              mma_f16_16x8x16_first(sum, a0, b0, a1, b1, x[n][b].x, x[n][b].y);
              mma_f16_16x8x16(sum, a2, b2, a3, b3, x[n][b].z, x[n][b].w);
              acc[n][0] = fmaf(sum[0], fa[b], acc[n][0]);
              acc[n][1] = fmaf(sum[1], fa[b], acc[n][1]);
              acc[n][2] = fmaf(sum[2], fb[b], acc[n][2]);
              acc[n][3] = fmaf(sum[3], fb[b], acc[n][3]);
            }
          }
        }
      }
      finish(sg, sg.tile + it - sg.item, ntiles, whole, acc);
    }
    const int runs = r.segments ? r.seg[r.segments - 1].run : 0;
    while (run < runs) restage(++run);  // (warps that have no unit in the last runs)
    cp_async_wait<0>();
  }
  __device__ void restage(int run) {
    __syncthreads();  // the columns staged before have been read
    stage(run);
    __syncthreads();
  }
};

// Step 5, all threads of the grid: a token's pairs added in their order.
__device__ void combine(const MoeParams& p) {
  const int64_t n = static_cast<int64_t>(p.T) * p.H;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * THREADS) {
    const int t = static_cast<int>(i / p.H), row = static_cast<int>(i - static_cast<int64_t>(t) * p.H);
    const float* src = p.part + static_cast<int64_t>(t) * p.top * p.H + row;
    float sum = 0.f;
#pragma unroll 4
    for (int k = 0; k < p.top; ++k) sum += __ldcg(src + static_cast<int64_t>(k) * p.H);
    p.y[t * p.ldy + row] = __float2bfloat16_rn(sum);
  }
}

template <int NT>
__global__ void __launch_bounds__(THREADS, 1) moe_mxfp4_kernel(const MoeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                             ~static_cast<uintptr_t>(127));
  __shared__ Routing r;
  float* red = reinterpret_cast<float*>(smem + RING_BYTES);
  uint8_t* staged = smem + RING_BYTES + WARPS * NT * 128 * 4;
  if (threadIdx.x == 0) r.abort = 0;
  route_start(p);
  if (grid_barrier(p, r, 1)) {
    route_choose(p, r);
    Product<NT, true>(p, r, staged, smem, red).run();
    __syncthreads();
    // (fetches its first weights, then waits for every h)
    Product<NT, false> down(p, r, staged, smem, red);
    if (grid_barrier(p, r, 2)) {
      down.run();
      if (grid_barrier(p, r, 3)) combine(p);
    }
    cp_async_wait<0>();
  }
  // The last CTA to leave clears the counters for the next call.
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(p.control + 1, 1u) == gridDim.x - 1) p.control[0] = p.control[1] = 0;
  }
}

template <int NT>
cudaError_t launch_t(MoeParams p, const DeviceCtl& ctl, cudaStream_t s) {
  constexpr int kSmem = 227 * 1024 - static_cast<int>(sizeof(Routing)) - 256;
  constexpr int kFixed = 128 + RING_BYTES + WARPS * NT * 128 * 4;
  auto kern = moe_mxfp4_kernel<NT>;
  const int pitch = (p.kt_h > p.kt_i ? p.kt_h : p.kt_i) * 256 + 64;
  p.stage_bytes = (kSmem - kFixed) / 16 * 16;
  if (p.stage_bytes < pitch) return cudaErrorInvalidValue;
  const int smem = kFixed + p.stage_bytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctl.sm_count);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_main_kernel("moe_mxfp4_kernel", ctl.sm_count, p.T * p.top);
  e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t moe_workspace(const MoeArgs& a, size_t (&at)[5]) {
  const size_t pairs = static_cast<size_t>(a.T) * a.top;
  size_t n = 0;
  auto take = [&](size_t bytes) {
    const size_t here = n;
    n += (bytes + 255) / 256 * 256;
    return here;
  };
  at[0] = take(static_cast<size_t>(a.T) * a.E * 4);
  at[1] = take(static_cast<size_t>(a.T) * 4);
  at[2] = take(pairs * 4);
  at[3] = take(pairs * scale_tiles(a.I) * 128 * 4);
  at[4] = take(pairs * a.H * 4);
  return n;
}

cudaError_t launch_moe(const MoeArgs& a, void* workspace, uint32_t* control, const DeviceCtl& ctl,
                       cudaStream_t s) {
  MoeParams p;
  p.x = static_cast<const __nv_bfloat16*>(a.x);
  p.router = static_cast<const __nv_bfloat16*>(a.router);
  p.ldx = a.ldx;
  p.ldr = a.ldr;
  p.up = a.up;
  p.up_s = a.up_scales;
  p.down = a.down;
  p.down_s = a.down_scales;
  p.ldu = a.ldu;
  p.ldd = a.ldd;
  p.y = static_cast<__nv_bfloat16*>(a.y);
  p.ldy = a.ldy;
  p.experts = a.experts;
  p.weights = a.weights;
  p.T = static_cast<int32_t>(a.T);
  p.E = static_cast<int32_t>(a.E);
  p.top = static_cast<int32_t>(a.top);
  p.H = static_cast<int32_t>(a.H);
  p.I = static_cast<int32_t>(a.I);
  p.kt_h = static_cast<int32_t>(scale_tiles(a.H));
  p.kt_i = static_cast<int32_t>(scale_tiles(a.I));
  size_t at[5];
  moe_workspace(a, at);
  char* ws = static_cast<char*>(workspace);
  p.logits = reinterpret_cast<float*>(ws + at[0]);
  p.x_mult = reinterpret_cast<float*>(ws + at[1]);
  p.h_max = reinterpret_cast<uint32_t*>(ws + at[2]);
  p.h = reinterpret_cast<float*>(ws + at[3]);
  p.part = reinterpret_cast<float*>(ws + at[4]);
  p.control = control;
  p.status = ctl.status;
  p.wait_limit_ns = ctl.wait_limit_ns;
  p.inject_stall = ctl.inject_stall;
  // an expert has at most T columns, and rarely more than 16: one or two tiles
  // of 8 at a time
  return a.T <= 8 ? launch_t<1>(p, ctl, s) : launch_t<2>(p, ctl, s);
}

}  // namespace mx
}  // namespace mhr
