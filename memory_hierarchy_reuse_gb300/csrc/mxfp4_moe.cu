// A whole mixture-of-experts layer for up to 64 tokens over 4-bit experts, in
// one launch:
//
//   logits = x R^T, the top experts of each token and their softmax weights,
//   h_p = silu(G_e x_t) * (U_e x_t)           for every chosen pair p = (t, e),
//   y_t = sum over p of weight_p D_e h_p.
//
// Bound by HBM: the chosen experts' weights pass once, 17/32 byte each, with a
// few multiply-adds a weight (as many as tokens chose the expert); the
// smallest calls by the latency of the dependent steps.  So one persistent
// cooperative grid, a CTA an SM, walks logits, the up product, h, the down
// product and the sum, with a grid barrier between each.
//
// The product.  Weights are the 128-row side of tcgen05.mma kind::mxf4 as they
// lie in memory: TMA moves their codes, and tcgen05.cp their scales, with no
// instruction spent on a weight (unpacking them in registers for mma.sync took
// some 200 issue slots per 16 x 128 weights and held the layer to 4.7 TB/s).
// That takes e2m1 columns too, so a column is written as a sum of eight: in each
// block of 32 the first is x over s = 2^ceil(log2(max / 6)) rounded to e2m1,
// and each further one the rest, over s / 4, s / 32, s / 256 and so on --
// after the first, whose largest values are 2 apart, the rest is at most 1 s,
// and after every other at most half its own unit.  The eighth leaves at most
// 2^-21 s, less than 2^-22 of the block's largest magnitude (or 2^-129, a quarter of
// the smallest scale, where that is more): what the fp32 sums
// lose is more (a model in 64 bits of 2048 x 768 with loud channels, before y's
// rounding: six / seven / eight terms 9e-6 / 1.1e-6 / 1.4e-7 of y, fp32 sums 6e-7).  The eight are columns
// of the MMA like any others, each with its own scales, and their fp32 sums are
// added in the epilogue: at this few columns the MMA's time is the reading of
// the 128 weight rows.  22 columns (176 of the MMA's N) are what two accumulators and
// the scales leave room for in TMEM.
//
// Work is cut into items of 128 weight rows x a part of K of one expert, and
// every CTA takes an equal run of them; the number of parts of K (up to 16) is
// picked so that the runs come out even.  A part's sums go to a buffer of
// their own, and whoever reads them adds the parts in order: results do not
// depend on the schedule.
//
// GB300, call after call: 64 tokens on 127 experts of 4096 x 1536 234 us (5.4 TB/s; 6.9
// while the products run, by stamps of six terms a column), 13 on 47 of 2600 x 1416 71
// us, 8 on 51 of 2048 x 768 45 us, one on 4 of 1024 x 512 18.5 us, of which the weights
// are one.  64 on 8 of 4096 x 1536, 16 pairs each: 53 us (six terms, 21 pairs an MMA: 49).  (A stage's MMAs are
// issued unrolled: with loops of a count known at run time only, a CTA took 0.41 us a
// stage, 43 GB/s, whatever the others did, and 64 tokens 253 us.)
#include "mhr_gemm.h"
#include "mhr_mxfp4.h"
#include "mxfp4_common.cuh"

namespace mhr {
namespace mx {
namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int CONSUMERS = THREADS - 32;        // all but warp 0, the producer
constexpr int TERMS = 8;                       // e2m1 columns a bf16 or fp32 column is written as
constexpr int MAX_COLS = 22;                   // columns an MMA takes at once, each TERMS of its N
constexpr int W_BYTES = 128 * 128;             // 128 rows x 256 columns of weights
constexpr int RING_STAGE = W_BYTES + 1024;     // and their scales
constexpr int STAGES = 6;
constexpr int RING_BYTES = STAGES * RING_STAGE;
constexpr int MAX_PAIRS = MOE_MAX_TOKENS * MOE_MAX_TOP;
constexpr int MAX_SEGMENTS = 272;
constexpr int PIECE = TERMS * (128 + 8);       // 256 columns of K as terms: codes, then scales
constexpr uint32_t ACC_COLS = MAX_COLS * TERMS;  // TMEM: two accumulators, scales of each stage
constexpr uint32_t SF_COL = 2 * ACC_COLS;
constexpr uint32_t SF_SET = 24;                // 128 rows of weights, up to 256 of columns
constexpr uint32_t TMEM_COLS = 512;
static_assert(SF_COL + STAGES * SF_SET <= TMEM_COLS, "scales fit");
static_assert(ACC_COLS <= 256 && TERMS == 8, "columns in groups of 8, scales in two tiles");
constexpr uint32_t kErrTimeoutGrid = 1u << 4;  // status word: a grid barrier's wait ran out

// One of the two products: rows of an expert in the packed matrix, K, and the
// partial sums it writes.
struct MoeProduct {
  const uint8_t* scales;
  int32_t rows;            // rows an expert has: 2 I or H
  int32_t tiles;           // tiles of 128 matrix rows that they can overlap
  int32_t blocks, kt, stages;  // of K: blocks of 32, scale tiles of 128, ring stages of 256
  float* sums;             // [part of K][pair][pitch]
  int32_t pitch;
};

// Tensor maps of the up and down weights: boxes of 128 rows, and of 32.
struct MoeMaps {
  CUtensorMap m[2][2];
};

struct MoeParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* router;
  int64_t ldx, ldr;
  __nv_bfloat16* y;
  int64_t ldy;
  int32_t* experts;
  float* weights;
  int32_t T, E, top, H, I;
  MoeProduct up, down;
  int32_t max_parts;       // of K
  // workspace
  float* logits;           // T x E
  uint8_t* x_terms;        // T x up.stages pieces
  uint8_t* h_terms;        // T * top x down.stages pieces
  uint32_t* control;       // [0] barrier arrivals, [1] exits
  int32_t stage_kb;        // shared memory for staged columns
  uint32_t* status;
  uint64_t wait_limit_ns;
  int32_t inject_stall;
};

// A CTA's run of items that share an expert, a part of K and their columns.
struct Segment {
  int16_t expert, first;          // pairs list[first .. first + count)
  uint8_t count, part;
  uint8_t k0, kn;                 // ring stages of K
  int16_t tile, items;            // tiles of 128 rows, from the expert's tile `tile` on
  int16_t run;                    // staged together with the others of its run
  uint16_t offset;                // of the staged columns in KB: scales, then codes

  __device__ int first_tile(const MoeProduct& m) const { return expert * m.rows / 128 + tile; }
};

struct Plan {
  int32_t segments, parts;
  Segment seg[MAX_SEGMENTS];
};

struct Routing {  // shared memory
  float weight[MAX_PAIRS];
  int16_t expert[MAX_PAIRS];      // of pair t * top + k
  int16_t list[MAX_PAIRS];        // pairs, expert by expert
  int32_t count[MOE_MAX_EXPERTS];    // pairs of an expert (zero but while they are sorted)
  int16_t offset[MOE_MAX_EXPERTS];   // its first place in list
  int16_t active[MOE_MAX_EXPERTS];   // the experts that some pair has
  int32_t num_active, most;          // and the most pairs that one has
  int4 warp[WARPS];                  // of 32 experts: pairs, active ones, most pairs
  Plan up, down;
};

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

// The chosen experts and weights of a token, by one warp; PER_LANE x 32 experts at
// most.  Logits become unsigned keys of the same order (a NaN largest, -0 and 0
// alike), 0 for one taken or none.  Lane k < top gets the k-th.
template <int PER_LANE>
__device__ __forceinline__ void choose_token(const MoeParams& p, int t, int& expert,
                                             float& weight) {
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
#pragma unroll 1
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
      expert = static_cast<int>(e);
    }
  }
  auto logit = [](uint32_t key) {
    return __uint_as_float(key == 0xffffffffu ? key : key >> 31 ? key & 0x7fffffffu : ~key);
  };
  weight = lane < p.top ? expf(logit(chosen) - logit(first)) : 0.f;
  float sum = weight;
#pragma unroll 1
  for (int d = 8; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  weight /= sum;
}

// Step 1, all warps of the grid: router logits, a warp one of them.
__device__ void route_logits(const MoeParams& p, int warp, int warps, bool vx, bool vr) {
  const int lane = threadIdx.x & 31;
  for (int task = warp; task < p.E * p.T; task += warps) {
    const int e = task / p.T, t = task - e * p.T;
    float sum = 0.f;
    for (int k = lane * 8; k - lane * 8 < p.H; k += 8 * 256) {
      uint4 w[8], x[8];
      load_row<8>(p.router + e * p.ldr, k, p.H, vr, w);
      load_row<8>(p.x + t * p.ldx, k, p.H, vx, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float wf[8], xf[8];
        unpack_bf16(w[i], wf);
        unpack_bf16(x[i], xf);
#pragma unroll
        for (int c = 0; c < 8; ++c) sum = fmaf(wf[c], xf[c], sum);
      }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) p.logits[t * p.E + e] = sum;
  }
}

// The same where there are more of them than warps: a CTA 16 tokens x 8 experts, its
// warps K in turns, added in their order.  On mma.sync (there is too little work for
// a tcgen05 tile's set-up): a lane's 8 columns of a row are its operands of two MMAs,
// of x and the router alike, whichever columns the MMA takes them for.
// GB300, a call with this and with a warp a logit: 24 tokens x 128 experts of 1024
// 28.7 / 31.9 us, 64 x 64 of 4096 57.3 / 57.4; fewer than the warps, 24 x 40 of 3000 45.3
// / 47.3, though with six terms a column 63.5 / 62.6.
__device__ void route_tiles(const MoeParams& p, float* parts, bool vx, bool vr) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2;
  const int sets = (p.T + 15) / 16, tiles = (p.E + 7) / 8 * sets;
#pragma unroll 1
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int e0 = tile / sets * 8, t0 = (tile - tile / sets * sets) * 16;
    const __nv_bfloat16* w = p.router + min(e0 + g, p.E - 1) * p.ldr;
    const __nv_bfloat16* x0 = p.x + min(t0 + g, p.T - 1) * p.ldx;
    const __nv_bfloat16* x1 = p.x + min(t0 + g + 8, p.T - 1) * p.ldx;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int k0 = (warp & 7) * 32 + (warp >> 3) * 1024; k0 < p.H; k0 += 2048) {
      const int k = k0 + (lane & 3) * 8;
      uint4 b[4], a0[4], a1[4];
      load_row<4>(w, k, p.H, vr, b);
      load_row<4>(x0, k, p.H, vx, a0);
      load_row<4>(x1, k, p.H, vx, a1);
      auto mma = [&](uint32_t p0, uint32_t p1, uint32_t p2, uint32_t p3, uint32_t q0, uint32_t q1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(sum[0]), "+f"(sum[1]), "+f"(sum[2]), "+f"(sum[3])
            : "r"(p0), "r"(p1), "r"(p2), "r"(p3), "r"(q0), "r"(q1));
      };
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mma(a0[i].x, a1[i].x, a0[i].y, a1[i].y, b[i].x, b[i].y);
        mma(a0[i].z, a1[i].z, a0[i].w, a1[i].w, b[i].z, b[i].w);
      }
    }
    float* mine = parts + warp * 128 + g * 8 + (lane & 3) * 2;
    mine[0] = sum[0], mine[1] = sum[1], mine[64] = sum[2], mine[65] = sum[3];
    __syncthreads();
    const int t = t0 + (threadIdx.x >> 3), e = e0 + (threadIdx.x & 7);
    if (threadIdx.x < 128 && t < p.T && e < p.E) {
      float all = 0.f;
#pragma unroll
      for (int i = 0; i < WARPS; ++i) all += parts[i * 128 + threadIdx.x];
      p.logits[t * p.E + e] = all;
    }
    __syncthreads();
  }
}

// 256 columns of K, 8 a lane, as TERMS rows of e2m1 codes and their scales, into a
// piece in memory (row j is 128 bytes from 128 j on, its 8 scales follow all rows)
// or, staged, into rows n on of a stage in shared memory (16-byte pieces
// swizzled by n % 8, scales in the tiles that tcgen05.cp takes).
//
// Here and below, code that runs twice a call is one copy of it, and loops stay
// rolled: between the grid barriers a CTA runs little code, and most of it for
// the first time in the launch, so that fetching instructions is what these steps
// wait for (choosing experts unrolled over four tokens took twice as long as one
// at a time).
__device__ __noinline__ void split_terms(float v0, float v1, float v2, float v3, float v4,
                                         float v5, float v6, float v7, uint8_t* codes,
                                         uint8_t* scales, int n, bool staged) {
  const int lane = threadIdx.x & 31, block = lane >> 2;
  float v[8] = {v0, v1, v2, v3, v4, v5, v6, v7};
  uint32_t amax = __float_as_uint(max_abs8(v));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  // the least power of two that is not below max / 6 = max / (1.5 * 4)
  const bool finite = amax < 0x7f800000u;  // else the block's scales are NaN
  int c = static_cast<int>(amax >> 23) - 2 + ((amax & 0x7fffffu) > 0x400000u ? 1 : 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = finite ? v[i] : 0.f;
#pragma unroll 1
  for (int j = 0; j < TERMS; ++j, ++n) {
    // (no unit is below 2^-127, code 0: the terms leave 2^-129 where that is more)
    const uint32_t code = static_cast<uint32_t>(max(c, 0));
    const float scale = __uint_as_float(code ? code << 23 : 1u << 22);
    const uint32_t word = encode8(v, __uint_as_float((254u - code) << 23));
    *reinterpret_cast<uint32_t*>(codes + n * 128 + ((block ^ (staged ? n & 7 : 0)) << 4) +
                                 (lane & 3) * 4) = word;
    if ((lane & 3) == 0)
      scales[staged ? (block >> 2) * 512 + (n & 31) * 16 + (n >> 5) * 4 + (block & 3)
                    : n * 8 + block] = static_cast<uint8_t>(finite ? code : 255u);
    const uint32_t h[4] = {e2m1_to_f16x2<0>(word), e2m1_to_f16x2<1>(word), e2m1_to_f16x2<2>(word),
                           e2m1_to_f16x2<3>(word)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // the rest: exact
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      v[2 * i] = fmaf(-f.x, scale, v[2 * i]);
      v[2 * i + 1] = fmaf(-f.y, scale, v[2 * i + 1]);
    }
    c -= j == 0 ? 2 : 3;
  }
}

// Whether each CTA makes the h that it needs as it stages it, or all of them are
// made once, between two barriers.  GB300, experts of 2048 x 768: 16 pairs 26.1 against
// 26.7 us a call, 32 pairs 30.8 / 30.7, 64 pairs of 8 tokens 43.4 / 43.1, of 32 tokens
// 45.9 / 45.1.  (Up to 16 pairs also keep to one scale tile a stage, as make_h has it.)
__device__ __forceinline__ bool direct_h(const MoeParams& p) { return p.T * p.top <= 16; }

// Step 1, all warps of the grid: x as terms, and the logits.
__device__ void route_start(const MoeParams& p, float* parts) {
  const int warp = (threadIdx.x >> 5) * gridDim.x + blockIdx.x;  // neighbours on other SMs
  const int warps = gridDim.x * WARPS;
  const bool vx = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ldx % 8 == 0;
  const bool vr = reinterpret_cast<uintptr_t>(p.router) % 16 == 0 && p.ldr % 8 == 0;
  const int lane = threadIdx.x & 31;
  for (int i = warps - 1 - warp; i < p.T * p.up.stages; i += warps) {  // the warps with fewest logits
    const int t = i / p.up.stages, k = (i - t * p.up.stages) * 256 + lane * 8;
    uint4 x[1];
    load_row<1>(p.x + t * p.ldx, k, p.H, vx, x);
    float v[8];
    unpack_bf16(x[0], v);
    uint8_t* piece = p.x_terms + static_cast<int64_t>(i) * PIECE;
    split_terms(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], piece, piece + TERMS * 128, 0,
                false);
  }
  if (p.E * p.T <= warps)
    route_logits(p, warp, warps, vx, vr);
  else
    route_tiles(p, parts, vx, vr);
}

// Step 2: the top experts of the tokens t0, t0 + step, ..., and their weights.
__device__ void choose_experts(const MoeParams& p, Routing& r, int t0, int step, bool write) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int t = t0; t < p.T; t += step) {
    int e;
    float w;
    if (p.E <= 128)
      choose_token<4>(p, t, e, w);
    else
      choose_token<MOE_MAX_EXPERTS / 32>(p, t, e, w);
    if (lane < p.top) {
      const int i = t * p.top + lane;
      r.expert[i] = static_cast<int16_t>(e);
      r.weight[i] = w;
      if (write) {
        p.experts[i] = e;
        p.weights[i] = w;
      }
    }
  }
}

// Step 2, in every CTA alike: the pairs sorted by expert.  Warp w has experts 32 w
// to 32 w + 31.
__device__ void sort_pairs(const MoeParams& p, Routing& r) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = threadIdx.x;
  static_assert(THREADS >= MOE_MAX_EXPERTS, "a thread an expert");
  const int pairs = p.T * p.top;
  // Up to 32 pairs by one warp, a lane a pair; experts in the order of their first
  // pairs.  GB300: 4 pairs 20.1 against 20.5 us a call, 32 pairs the same as below.
  if (pairs <= 32) {
    if (warp == 0) {
      const int x = lane < pairs ? r.expert[lane] : -1 - lane;
      const uint32_t same = __match_any_sync(0xffffffffu, x), before = (1u << lane) - 1;
      const bool first = lane < pairs && (same & before) == 0;
      const uint32_t firsts = __ballot_sync(0xffffffffu, first);
      const int count = __popc(same);
      int scan = first ? count : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += o;
      }
      // the first pair's lane holds its expert's place in the list
      const int offset = __shfl_sync(0xffffffffu, scan - count, __ffs(same) - 1);
      if (first) {
        r.offset[x] = static_cast<int16_t>(offset);
        r.active[__popc(firsts & before)] = static_cast<int16_t>(x);
      }
      if (lane < pairs) r.list[offset + __popc(same & before)] = static_cast<int16_t>(lane);
      const int most = __reduce_max_sync(0xffffffffu, first ? count : 0);
      if (lane == 0) {
        r.num_active = __popc(firsts);
        r.most = most;
      }
    }
    __syncthreads();
    return;
  }
  for (int i = threadIdx.x; i < pairs; i += THREADS) atomicAdd(&r.count[r.expert[i]], 1);
  __syncthreads();
  const int count = e < p.E ? r.count[e] : 0;
  const uint32_t has = __ballot_sync(0xffffffffu, count > 0);
  int scan = count;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, scan, d);
    if (lane >= d) scan += o;
  }
  const int most = __reduce_max_sync(0xffffffffu, count);
  if (lane == 31) r.warp[warp] = make_int4(scan, __popc(has), most, 0);
  __syncthreads();
  // the warps before this one: pairs, active experts
  const int4 w = lane < WARPS ? r.warp[lane] : make_int4(0, 0, 0, 0);
  const int offset = __reduce_add_sync(0xffffffffu, lane < warp ? w.x : 0);
  const int active = __reduce_add_sync(0xffffffffu, lane < warp ? w.y : 0);
  if (count > 0) {
    r.offset[e] = static_cast<int16_t>(offset + scan - count);
    r.active[active + __popc(has & ((1u << lane) - 1))] = static_cast<int16_t>(e);
  }
  if (warp == 0) {
    const int all = __reduce_add_sync(0xffffffffu, w.y), top = __reduce_max_sync(0xffffffffu, w.z);
    if (lane == 0) {
      r.num_active = all;
      r.most = top;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += THREADS) {
    const int x = r.expert[i];
    // an expert's pairs, from its list's end down, in any order: each is a
    // column of its own (this takes count to zero)
    r.list[r.offset[x] + atomicSub(&r.count[x], 1) - 1] = static_cast<int16_t>(i);
  }
  __syncthreads();
}

// KB that `cols` columns over `stages` stages of K take when staged -- a stage's
// scale tiles, 1 KB for each 128 rows, then 128 bytes a row and stage -- and how many
// columns fit into `kb` KB.
__device__ __forceinline__ int staged_rows(int cols) { return cols * TERMS; }
__device__ __forceinline__ int scales_kb(int cols) { return cols > 128 / TERMS ? 2 : 1; }
__device__ __forceinline__ int staged_kb(int cols, int stages) {
  return stages * (scales_kb(cols) + cols);
}
__host__ __device__ __forceinline__ int columns_that_fit(int kb, int stages) {
  const int one = kb / stages - 1, n = one > 128 / TERMS ? one - 1 : one;
  return n < MAX_COLS ? n : MAX_COLS;
}

// By one warp: the parts of K, then the CTA's equal run of all items -- expert by
// expert, part by part, tile by tile -- as segments.  An expert's items are taken
// again when more pairs have it than fit an MMA or shared memory, and segments are
// staged together as far as they fit.
__device__ void plan_product(const MoeParams& p, const MoeProduct& m, const Routing& r, Plan& plan) {
  const int lane = threadIdx.x & 31;
  const int pairs = p.T * p.top, active = r.num_active;
  auto end_of = [&](int ai) {
    return ai + 1 < active ? static_cast<int>(r.offset[r.active[ai + 1]]) : pairs;
  };
  // Time of the longest run, in stages, with half of one for an item's ends (GB300:
  // with a quarter, 2 tokens on 7 experts of 2048 x 1024 took 26.6 us instead of
  // 22.6, 64 tokens with one each of 59 of 4096 x 256 39.0 instead of 37.1), times the passes that
  // the expert with the most pairs takes.  (One column at a
  // time serves experts of one pair only: MAX_SEGMENTS counts on two, which fit 2
  // parts of any K.)
  const int parts = lane + 1;
  uint32_t cost = 0xffffffffu;
  if (parts <= p.max_parts && parts <= m.stages) {
    const uint32_t items = static_cast<uint32_t>(active) * parts * m.tiles;
    const uint32_t longest = (items + gridDim.x - 1) / gridDim.x;
    const int stages = (m.stages + parts - 1) / parts;
    const int fit = columns_that_fit(p.stage_kb, stages);
    if (fit >= min(r.most, 2)) {
      cost = longest * (2 * stages + 1) * ((r.most + fit - 1) / fit);
      cost = min(cost, 0x7fffffeu) * 32 + lane;  // ties: the fewest parts
    }
  }
  const int chosen = static_cast<int>(__reduce_min_sync(0xffffffffu, cost) & 31u) + 1;
  if (lane == 0) {
    const int fit = columns_that_fit(p.stage_kb, (m.stages + chosen - 1) / chosen);
    const uint32_t items = static_cast<uint32_t>(active) * chosen * m.tiles;
    // (at most 512 experts x 16 parts x 258 tiles x some hundred CTAs: 32 bits)
    const int begin = static_cast<int>(items * blockIdx.x / gridDim.x);
    const int end = static_cast<int>(items * (blockIdx.x + 1) / gridDim.x);
    int n = 0, run = 0, offset = 0;
    for (int u = begin; u < end;) {
      const int row = u / m.tiles, t = u - row * m.tiles;
      const int ai = row / chosen, part = row - ai * chosen, e = r.active[ai];
      const int items = min(m.tiles - t, end - u);
      u += items;
      const int64_t r0 = static_cast<int64_t>(e) * m.rows;
      const int tile0 = static_cast<int>(r0 / 128);
      const int tiles = min(items, static_cast<int>((r0 + m.rows - 1) / 128) + 1 - (tile0 + t));
      if (tiles <= 0) continue;
      const int k0 = m.stages * part / chosen, k1 = m.stages * (part + 1) / chosen;
      for (int c = r.offset[e]; c < end_of(ai); c += fit) {
        const int count = min(fit, end_of(ai) - c), kb = staged_kb(count, k1 - k0);
        if (offset + kb > p.stage_kb) {
          ++run;
          offset = 0;
        }
        Segment& s = plan.seg[n++];
        s.expert = static_cast<int16_t>(e);
        s.first = static_cast<int16_t>(c);
        s.count = static_cast<uint8_t>(count);
        s.part = static_cast<uint8_t>(part);
        s.k0 = static_cast<uint8_t>(k0);
        s.kn = static_cast<uint8_t>(k1 - k0);
        s.tile = static_cast<int16_t>(t);
        s.items = static_cast<int16_t>(tiles);
        s.run = static_cast<int16_t>(run);
        s.offset = static_cast<uint16_t>(offset);
        offset += kb;
      }
    }
    plan.segments = n;
    plan.parts = chosen;
  }
}

// Everything the warps of a CTA share.
struct Cta {
  const MoeParams& p;
  Routing& r;
  volatile int* abort_flag;
  uint8_t* staged;
  uint32_t ring, bar0, tmem;
  int warp, lane;
  uint32_t it, ph_items;  // of this warp's role: ring stages, items

  __device__ uint32_t full_bar(uint32_t s) const { return bar0 + 8u * s; }
  __device__ uint32_t empty_bar(uint32_t s) const { return bar0 + 8u * (STAGES + s); }
  __device__ uint32_t acc_full(uint32_t b) const { return bar0 + 8u * (2 * STAGES + b); }
  __device__ uint32_t acc_empty(uint32_t b) const { return bar0 + 8u * (2 * STAGES + 2 + b); }
  __device__ void give_up(uint32_t bit) const {  // by one thread
    if (!*abort_flag) atomicOr(p.status, bit);
    *abort_flag = 1;
  }
  __device__ bool wait(uint32_t bar, uint32_t parity, uint32_t bit) const {  // by a warp
    const bool ok = __all_sync(
        0xffffffffu, mbar_wait_bounded(bar, parity, p.wait_limit_ns, abort_flag)) != 0;
    if (!ok && lane == 0) give_up(bit);
    __syncwarp();
    return ok;
  }
};

__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(CONSUMERS) : "memory");
}

// All CTAs of the (cooperative) grid, by the consumer warps; bounded.
__device__ __forceinline__ void grid_barrier(const Cta& c, uint32_t round) {
  consumers_sync();
  if (threadIdx.x == 32 && !*c.abort_flag) {
    __threadfence();
    const bool absent = c.p.inject_stall && blockIdx.x == 0 && round == 1;  // test hook
    if (!absent) atomicAdd(c.p.control, 1u);
    const uint32_t want = round * gridDim.x;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t n = 1;; ++n) {
      uint32_t arrived;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];"
                   : "=r"(arrived)
                   : "l"(c.p.control)
                   : "memory");
      if (arrived >= want) break;
      if ((n & 63u) == 0 && global_timer_ns() - t0 > c.p.wait_limit_ns) {
        c.give_up(kErrTimeoutGrid);
        break;
      }
    }
  }
  consumers_sync();
}

// The weights of a plan's items, into the ring.  By one warp, converged.  A tile
// that reaches past the expert's rows brings those of its quarters that hold
// some: an expert's rows start and end anywhere in the matrix' tiles of 128, to
// which the scales' tiles tie the MMA's rows (60 experts of 2 x 1416 rows: 8 %
// fewer bytes than with whole tiles).
__device__ __forceinline__ bool produce(Cta& c, const CUtensorMap* whole,
                                        const CUtensorMap* quarter, const MoeProduct& m,
                                        const Plan& plan) {
  uint32_t st = c.it % STAGES, ph = (c.it / STAGES) & 1u;
  for (int s = 0; s < plan.segments; ++s) {
    const Segment sg = plan.seg[s];
    const int row0 = sg.expert * m.rows, row1 = row0 + m.rows;
    const int t0 = sg.first_tile(m);
    for (int t = t0; t < t0 + sg.items; ++t) {
      // quarters [q0, q1) of the tile
      const int q0 = max(row0 - t * 128, 0) >> 5, q1 = min(row1 - t * 128 + 31, 128) >> 5;
      for (int k = sg.k0; k < sg.k0 + sg.kn; ++k) {
        if (!__all_sync(0xffffffffu, mbar_try_wait(c.empty_bar(st), ph ^ 1u)) &&
            !c.wait(c.empty_bar(st), ph ^ 1u, kErrTimeoutProducer))
          return false;
        const uint32_t bytes = static_cast<uint32_t>(min(2, m.kt - 2 * k)) * 512u;
        const uint32_t at = c.ring + st * RING_STAGE;
        if (elect_one()) {
          mbar_arrive_expect_tx(c.full_bar(st), (q1 - q0) * (W_BYTES / 4) + bytes);
          if (q1 - q0 == 4)
            tma_load_2d(at, whole, c.full_bar(st), k * 128, t * 128);
          else
            for (int q = q0; q < q1; ++q)
              tma_load_2d(at + q * (W_BYTES / 4), quarter, c.full_bar(st), k * 128,
                          t * 128 + q * 32);
          bulk_load(at + W_BYTES, m.scales + (static_cast<int64_t>(t) * m.kt + 2 * k) * 512, bytes,
                    c.full_bar(st));
        }
        __syncwarp();
        ++c.it;
        if (++st == STAGES) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
  }
  return true;
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// The columns of a run's segments into shared memory, by the consumer warps, all
// copies under way at once: of each pair and stage of 256 columns of K, TERMS
// rows of 8 pieces of 16 bytes (row n's swizzled by n % 8), and their scales as
// words of 4 into the tiles that tcgen05.cp takes.
__device__ __forceinline__ void stage_columns(const Cta& c, const MoeProduct& m, const Plan& plan, bool up,
                              int run) {
  const MoeParams& p = c.p;
  static_assert(TERMS * 10 <= 96, "three copies a lane");
  for (int s = 0; s < plan.segments; ++s) {
    const Segment sg = plan.seg[s];
    if (sg.run != run) continue;
    const int rows = staged_rows(sg.count), stage_scales = scales_kb(sg.count) * 1024;
    const uint32_t scales = smem_u32(c.staged) + sg.offset * 1024,
                   codes = scales + sg.kn * stage_scales;
    for (int i = c.warp - 1; i < sg.count * sg.kn; i += CONSUMERS / 32) {  // a pair's stage a warp
      const int col = i / sg.kn, stage = i - col * sg.kn;
      const int pair = c.r.list[sg.first + col];
      const uint8_t* src =
          (up ? p.x_terms : p.h_terms) +
          (static_cast<int64_t>(up ? pair / p.top : pair) * m.stages + sg.k0 + stage) * PIECE;
#pragma unroll
      for (int copy = c.lane; copy < 96; copy += 32) {  // 8 pieces and 2 words a row
        if (copy < TERMS * 8) {
          const int n = col * TERMS + (copy >> 3), block = copy & 7;
          cp_async_16(codes + (stage * rows + n) * 128 + ((block ^ (n & 7)) << 4), src + copy * 16);
        } else if (copy < TERMS * 10) {
          const int w = copy - TERMS * 8, n = col * TERMS + (w >> 1);
          cp_async_4(scales + stage * stage_scales + (n >> 7) * 1024 + (w & 1) * 512 +
                         (n & 31) * 16 + (n >> 5 & 3) * 4,
                     src + TERMS * 128 + w * 4);
        }
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// h of a pair for 8 columns from k on: the parts' sums of gate and up in their
// order.  (expf and a division: the error of the fast exponential grows with the
// gate's magnitude, some 30 units in the last place of silu at -80.)
__device__ __forceinline__ void h_of(const Cta& c, int pair, int k, float (&h)[8]) {
  const MoeParams& p = c.p;
  const int64_t part = static_cast<int64_t>(p.T) * p.top * p.up.pitch;
  const int half = p.up.pitch / 2;
  const float* g = p.up.sums + static_cast<int64_t>(pair) * p.up.pitch + k;
  float gate[8], value[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) gate[j] = value[j] = 0.f;
  if (k < p.I)
#pragma unroll 1
    for (int q = 0; q < c.r.up.parts; q += 2) {  // two at once
      const bool both = q + 1 < c.r.up.parts;
      float4 a[2][2], b[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float* at = g + (i && both ? part : 0);
        a[i][0] = __ldcg(reinterpret_cast<const float4*>(at));
        a[i][1] = __ldcg(reinterpret_cast<const float4*>(at) + 1);
        b[i][0] = __ldcg(reinterpret_cast<const float4*>(at + half));
        b[i][1] = __ldcg(reinterpret_cast<const float4*>(at + half) + 1);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i && !both) break;
        gate[0] += a[i][0].x, gate[1] += a[i][0].y, gate[2] += a[i][0].z, gate[3] += a[i][0].w;
        gate[4] += a[i][1].x, gate[5] += a[i][1].y, gate[6] += a[i][1].z, gate[7] += a[i][1].w;
        value[0] += b[i][0].x, value[1] += b[i][0].y, value[2] += b[i][0].z, value[3] += b[i][0].w;
        value[4] += b[i][1].x, value[5] += b[i][1].y, value[6] += b[i][1].z, value[7] += b[i][1].w;
      }
      g += 2 * part;
    }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    h[j] = k + j < p.I ? gate[j] / (1.f + expf(-gate[j])) * value[j] : 0.f;
}

// h of some pairs as terms, 256 columns a warp: of all pairs into memory, by the
// consumers of the grid (run < 0), or of a run's segments straight into shared
// memory, by this CTA's.
__device__ __forceinline__ void make_h(const Cta& c, const Plan& plan, int run) {
  const MoeParams& p = c.p;
  const int stages = p.down.stages;
  constexpr int TEAM = CONSUMERS / 32;
  const int segments = run < 0 ? 1 : plan.segments;
#pragma unroll 1
  for (int s = 0; s < segments; ++s) {
    if (run >= 0 && plan.seg[s].run != run) continue;
    const int first = run < 0 ? (c.warp - 1) * gridDim.x + blockIdx.x : c.warp - 1;
    const int step = run < 0 ? TEAM * gridDim.x : TEAM;
    const int k0 = run < 0 ? 0 : plan.seg[s].k0, kn = run < 0 ? stages : plan.seg[s].kn;
    const int tasks = run < 0 ? p.T * p.top * stages : plan.seg[s].count * kn;
#pragma unroll 1
    for (int i = first; i < tasks; i += step) {
      const int col = i / kn, stage = i - col * kn;
      const int pair = run < 0 ? col : c.r.list[plan.seg[s].first + col];
      float h[8];
      h_of(c, pair, (k0 + stage) * 256 + c.lane * 8, h);
      uint8_t *codes, *scales;
      if (run < 0) {
        codes = p.h_terms + static_cast<int64_t>(i) * PIECE;
        scales = codes + TERMS * 128;
      } else {
        uint8_t* at = c.staged + plan.seg[s].offset * 1024;
        codes = at + kn * 1024 + stage * staged_rows(plan.seg[s].count) * 128;  // (up to 16 pairs)
        scales = at + stage * 1024;
      }
      split_terms(h[0], h[1], h[2], h[3], h[4], h[5], h[6], h[7], codes, scales,
                  run < 0 ? 0 : col * TERMS, run >= 0);
    }
  }
}

// The MMAs of a segment, by one warp.
__device__ __forceinline__ bool multiply(Cta& c, const MoeProduct& m, const Segment& sg) {
  const int rows = staged_rows(sg.count);
  const uint32_t id0 = make_idesc_mxf4(128, rows, 0), id2 = make_idesc_mxf4(128, rows, 2);
  // above 128 rows: two scale tiles for every 128 columns of K, 1 KB apart in a stage
  const bool two = scales_kb(sg.count) == 2;
  const uint32_t stage_scales = (two ? 2048 : 1024) >> 4, sf_k = two ? 8 : 4;
  const uint32_t scales = desc_lo(smem_u32(c.staged) + sg.offset * 1024);
  const uint32_t codes = scales + sg.kn * stage_scales;
  uint32_t st = c.it % STAGES, ph = (c.it / STAGES) & 1u;
  for (int t = 0; t < sg.items; ++t, ++c.ph_items) {
    const uint32_t b = c.ph_items & 1u;
    if (!c.wait(c.acc_empty(b), ((c.ph_items >> 1) & 1u) ^ 1u, kErrTimeoutMma)) return false;
    tc_fence_after();
    const uint32_t d = c.tmem + b * ACC_COLS;
    for (int k = 0; k < sg.kn; ++k) {
      // (a stage's scales have TMEM columns of their own: whoever read them last
      // had finished before the producer filled the stage again)
      if (!__all_sync(0xffffffffu, mbar_try_wait(c.full_bar(st), ph)) &&
          !c.wait(c.full_bar(st), ph, kErrTimeoutMma))
        return false;
      tc_fence_after();
      const uint32_t w = desc_lo(c.ring + st * RING_STAGE), cw = w + (W_BYTES >> 4);
      const uint32_t x = codes + k * rows * (128 >> 4), cx = scales + k * stage_scales;
      const uint32_t sfw = c.tmem + SF_COL + st * SF_SET, sfx = sfw + 8;
      const int left = m.blocks - (sg.k0 + k) * 8;
      const uint32_t first = k > 0 ? 1u : 0u;
      if (elect_one()) {
        if (left >= 8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            copy_scale_tile<1>(sfw + 4 * i, cw + 32 * i);
            copy_scale_tile<1>(sfx + sf_k * i, cx + 32 * i);
            if (two) copy_scale_tile<1>(sfx + sf_k * i + 4, cx + 64 + 32 * i);
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_mxf4<1>(d, w + 2 * kk, x + 2 * kk, kk & 1 ? id2 : id0, sfw + 4 * (kk >> 1),
                        sfx + sf_k * (kk >> 1), kk > 0 ? 1u : first);
        } else {  // the last stage of K
          const int kts = left > 4 ? 2 : 1, mmas = (left + 1) / 2;
          for (int i = 0; i < kts; ++i) {
            copy_scale_tile<1>(sfw + 4 * i, cw + 32 * i);
            copy_scale_tile<1>(sfx + sf_k * i, cx + 32 * i);
            if (two) copy_scale_tile<1>(sfx + sf_k * i + 4, cx + 64 + 32 * i);
          }
          for (int kk = 0; kk < mmas; ++kk)
            mma_mxf4<1>(d, w + 2 * kk, x + 2 * kk, kk & 1 ? id2 : id0, sfw + 4 * (kk >> 1),
                        sfx + sf_k * (kk >> 1), kk > 0 ? 1u : first);
        }
        mma_commit(c.empty_bar(st));
        if (k + 1 == sg.kn) mma_commit(c.acc_full(b));
      }
      __syncwarp();
      ++c.it;
      if (++st == STAGES) {
        st = 0;
        ph ^= 1u;
      }
    }
  }
  return true;
}

// A segment's sums out of TMEM: the terms of a column added, smallest first, one
// matrix row a lane.  By four warps.
__device__ __forceinline__ bool write_sums(Cta& c, const MoeProduct& m, const Segment& sg, bool up) {
  const int q = c.warp & 3;
  const int pairs = c.p.T * c.p.top;
  const int row0 = sg.first_tile(m) * 128 - sg.expert * m.rows + q * 32 + c.lane;  // of the expert
  for (int t = 0; t < sg.items; ++t, ++c.ph_items) {
    const uint32_t b = c.ph_items & 1u;
    if (!c.wait(c.acc_full(b), (c.ph_items >> 1) & 1u, kErrTimeoutEpilogue)) return false;
    tc_fence_after();
    const uint32_t taddr = c.tmem + b * ACC_COLS + (static_cast<uint32_t>(q * 32) << 16);
    const int row = row0 + t * 128;
    const bool in = row >= 0 && row < m.rows;
    // up: gate rows, then up rows at half the pitch
    const int at = up && row >= c.p.I ? row - c.p.I + m.pitch / 2 : row;
    float* sums = m.sums + static_cast<int64_t>(sg.part) * pairs * m.pitch + at;
    for (int c0 = 0; c0 < sg.count; c0 += 4) {  // 4 columns: 32 TMEM columns
      uint32_t v[TERMS / 2][8];
#pragma unroll
      for (int i = 0; i < TERMS / 2; ++i) tmem_ld_8cols(taddr + c0 * TERMS + 8 * i, v[i]);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float sum = 0.f;
#pragma unroll
        for (int i = TERMS - 1; i >= 0; --i)
          sum += __uint_as_float(v[(j * TERMS + i) / 8][(j * TERMS + i) % 8]);
        if (in && c0 + j < sg.count)
          sums[static_cast<int64_t>(c.r.list[sg.first + c0 + j]) * m.pitch] = sum;
      }
    }
    tc_fence_before();
    __syncwarp();
    if (c.lane == 0) mbar_arrive(c.acc_empty(b));
  }
  return true;
}

// Steps 3 and 4, by the consumer warps.
__device__ __forceinline__ void product(Cta& c, const MoeProduct& m, const Plan& plan, bool up) {
  const int runs = plan.segments ? plan.seg[plan.segments - 1].run + 1 : 0;
  int s = 0;
  for (int run = 0; run < runs; ++run) {
    if (run) consumers_sync();  // the columns staged before have been read
    if (!*c.abort_flag) {
      if (!up && direct_h(c.p))
        make_h(c, plan, run);
      else
        stage_columns(c, m, plan, up, run);
    }
    fence_proxy_async_smem();
    consumers_sync();
    bool ok = !*c.abort_flag;
    for (; s < plan.segments && plan.seg[s].run == run; ++s) {
      if (!ok) continue;
      if (c.warp == 1) {
        ok = multiply(c, m, plan.seg[s]);
      } else if (c.warp >= 4 && c.warp < 8) {
        ok = write_sums(c, m, plan.seg[s], up);
      }
    }
    // The MMA warp waits for its own, which read the staged columns.
    if (c.warp == 1 && ok && c.it > 0)
      c.wait(c.empty_bar((c.it - 1) % STAGES), ((c.it - 1) / STAGES) & 1u, kErrTimeoutMma);
  }
}

// Step 5, the consumers of the grid: a token's pairs added, four rows for four
// lanes, which take every fourth pair each.
__device__ __forceinline__ void combine(const Cta& c) {
  const MoeParams& p = c.p;
  const int quads = (p.H + 3) / 4, n = p.T * quads * 4;
  const int64_t part = static_cast<int64_t>(p.T) * p.top * p.down.pitch;
  const int parts = c.r.down.parts, sub = c.lane & 3;
  const int loads = (p.top - sub + 3) / 4 * parts;
  for (int i = blockIdx.x * CONSUMERS + threadIdx.x - 32; i - c.lane < n;
       i += gridDim.x * CONSUMERS) {
    const int at = min(i, n - 1) >> 2, t = at / quads, row = (at - t * quads) * 4;
    const float* src = p.down.sums + static_cast<int64_t>(t) * p.top * p.down.pitch + row;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    // a pair's parts are added first; eight loads are under way at once
    float pair[4] = {0.f, 0.f, 0.f, 0.f};
    int k = sub, q = 0;  // pair and part of the load to be added
#pragma unroll 1
    for (int l0 = 0; l0 < loads; l0 += 8) {
      float4 v[8];
      int lk = k, lq = q;  // pair and part of the load
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (l0 + j >= loads) break;
        v[j] = __ldcg(reinterpret_cast<const float4*>(src + static_cast<int64_t>(lk) * p.down.pitch +
                                                      lq * part));
        if (++lq == parts) {
          lq = 0;
          lk += 4;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (l0 + j >= loads) break;
        pair[0] += v[j].x, pair[1] += v[j].y, pair[2] += v[j].z, pair[3] += v[j].w;
        if (++q == parts) {
          const float w = c.r.weight[t * p.top + k];
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            sum[i4] = fmaf(w, pair[i4], sum[i4]);
            pair[i4] = 0.f;
          }
          q = 0;
          k += 4;
        }
      }
    }
    __syncwarp();
    float y = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 1);
      sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 2);
      if (sub == j) y = sum[j];
    }
    if (i < n && row + sub < p.H) p.y[t * p.ldy + row + sub] = __float2bfloat16_rn(y);
  }
}

__global__ void __launch_bounds__(THREADS, 1)
    moe_mxfp4_kernel(const __grid_constant__ MoeMaps maps,
                     const __grid_constant__ MoeParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Routing r;
  __shared__ alignas(8) uint64_t bars[2 * STAGES + 4];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Cta c{p, r, &abort_flag, smem + RING_BYTES, smem_u32(smem), smem_u32(bars), 0,
        static_cast<int>(threadIdx.x >> 5), static_cast<int>(threadIdx.x & 31), 0, 0};
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(c.full_bar(s), 1);
      mbar_init(c.empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(c.acc_full(b), 1);
      mbar_init(c.acc_empty(b), 4);
    }
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.m[0][0]);
    tma_prefetch_desc(&maps.m[1][0]);
  }
  if (c.warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  for (int e = threadIdx.x; e < p.E; e += THREADS) r.count[e] = 0;
  route_start(p, reinterpret_cast<float*>(c.staged));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  c.tmem = tmem_slot;
  if (c.warp) grid_barrier(c, 1);
  __syncthreads();
  uint32_t round = 2;
  if (p.T <= WARPS) {  // every CTA chooses for all tokens, a warp one token
    if (!abort_flag) choose_experts(p, r, c.warp, WARPS, blockIdx.x == 0);
  } else {
    // a warp of the grid each, then a barrier (64 tokens in every CTA took 5.4 us)
    if (!abort_flag && c.warp)
      choose_experts(p, r, blockIdx.x + (c.warp - 1) * gridDim.x, CONSUMERS / 32 * gridDim.x, true);
    if (c.warp) grid_barrier(c, round++);
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * p.top && !abort_flag; i += THREADS) {
      r.expert[i] = static_cast<int16_t>(__ldcg(p.experts + i));
      r.weight[i] = __ldcg(p.weights + i);
    }
  }
  __syncthreads();
  if (!abort_flag) {
    sort_pairs(p, r);
    if (c.warp == 0) plan_product(p, p.up, r, r.up);
    if (c.warp == 1) plan_product(p, p.down, r, r.down);
  } else if (threadIdx.x == 0) {
    r.up.segments = r.down.segments = 0;
  }
  __syncthreads();
  if (c.warp == 0) {
    // The producer runs ahead through both products: weights wait for nothing
    // but their place in the ring.
    bool ok = true;
#pragma unroll 1
    for (int i = 0; ok && i < 2; ++i)
      ok = produce(c, &maps.m[i][0], &maps.m[i][1], i ? p.down : p.up, i ? r.down : r.up);
    if (c.lane == 0) {
      volatile int never = 0;  // its copies in flight have landed before it leaves
      for (uint32_t i = c.it > STAGES ? c.it - STAGES : 0; i < c.it; ++i)
        if (!mbar_wait_bounded(c.full_bar(i % STAGES), (i / STAGES) & 1u, p.wait_limit_ns, &never))
          atomicOr(p.status, kErrTimeoutDrain);
    }
    __syncwarp();
  } else {
    // up, barrier, h, barrier; down, barrier, sum
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      product(c, i ? p.down : p.up, i ? r.down : r.up, i == 0);
      grid_barrier(c, round++);
      if (i == 0) {
        if (direct_h(p)) continue;
        if (!abort_flag) make_h(c, r.down, -1);
        grid_barrier(c, round++);
      } else {
        // No CTA polls any more once it is here: the last one clears the counters
        // for the next call.
        if (threadIdx.x == 32 && atomicAdd(p.control + 1, 1u) == gridDim.x - 1)
          p.control[0] = p.control[1] = 0;
        if (!abort_flag) combine(c);
      }
    }
    if (c.warp == 1 && c.it > 0) {  // the last MMAs issued have finished
      volatile int never = 0;
      if (!mbar_wait_bounded(c.empty_bar((c.it - 1) % STAGES), ((c.it - 1) / STAGES) & 1u,
                             p.wait_limit_ns, &never) && c.lane == 0)
        atomicOr(p.status, kErrTimeoutDrain);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (c.warp == 1) {
    tc_fence_after();
    tmem_dealloc(c.tmem, TMEM_COLS);
  }
}

int max_parts(int64_t pairs) {  // of K: the partial sums' memory
  const int64_t n = 2048 / pairs;
  return static_cast<int>(n < 2 ? 2 : n > 16 ? 16 : n);
}
int64_t up_pitch(int64_t I) { return 2 * ((I + 7) / 8 * 8); }
int64_t down_pitch(int64_t H) { return (H + 3) / 4 * 4; }

}  // namespace

size_t moe_workspace(const MoeArgs& a, size_t (&at)[5]) {
  const int64_t pairs = a.T * a.top;
  size_t n = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = n;
    n += (static_cast<size_t>(bytes) + 255) / 256 * 256;
    return here;
  };
  at[0] = take(a.T * a.E * 4);
  at[1] = take(max_parts(pairs) * pairs * up_pitch(a.I) * 4);
  at[2] = take(max_parts(pairs) * pairs * down_pitch(a.H) * 4);
  at[3] = take(a.T * ((scale_tiles(a.H) + 1) / 2) * PIECE);
  at[4] = take(pairs * ((scale_tiles(a.I) + 1) / 2) * PIECE);
  return n;
}

cudaError_t launch_moe(const MoeArgs& a, void* workspace, uint32_t* control, const DeviceCtl& ctl,
                       cudaStream_t s) {
  MoeParams p;
  p.x = static_cast<const __nv_bfloat16*>(a.x);
  p.router = static_cast<const __nv_bfloat16*>(a.router);
  p.ldx = a.ldx;
  p.ldr = a.ldr;
  p.y = static_cast<__nv_bfloat16*>(a.y);
  p.ldy = a.ldy;
  p.experts = a.experts;
  p.weights = a.weights;
  p.T = static_cast<int32_t>(a.T);
  p.E = static_cast<int32_t>(a.E);
  p.top = static_cast<int32_t>(a.top);
  p.H = static_cast<int32_t>(a.H);
  p.I = static_cast<int32_t>(a.I);
  p.max_parts = max_parts(a.T * a.top);
  size_t at[5];
  moe_workspace(a, at);
  char* ws = static_cast<char*>(workspace);
  auto product_of = [&](const uint8_t* scales, int64_t rows, int64_t K, size_t sums, int64_t pitch) {
    MoeProduct m;
    m.scales = scales;
    m.rows = static_cast<int32_t>(rows);
    // an expert's rows may start anywhere in a tile, unless they are whole tiles
    m.tiles = static_cast<int32_t>(rows % 128 == 0 ? rows / 128 : (rows - 1 + 127) / 128 + 1);
    m.blocks = static_cast<int32_t>(blocks_of(K));
    m.kt = static_cast<int32_t>(scale_tiles(K));
    m.stages = (m.kt + 1) / 2;
    m.sums = reinterpret_cast<float*>(ws + sums);
    m.pitch = static_cast<int32_t>(pitch);
    return m;
  };
  p.up = product_of(a.up_scales, 2 * a.I, a.H, at[1], up_pitch(a.I));
  p.down = product_of(a.down_scales, a.H, a.I, at[2], down_pitch(a.H));
  p.logits = reinterpret_cast<float*>(ws + at[0]);
  p.x_terms = reinterpret_cast<uint8_t*>(ws + at[3]);
  p.h_terms = reinterpret_cast<uint8_t*>(ws + at[4]);
  p.control = control;
  p.status = ctl.status;
  p.wait_limit_ns = ctl.wait_limit_ns;
  p.inject_stall = ctl.inject_stall;
  MoeMaps maps;
  for (int i = 0; i < 4; ++i) {
    const bool down = i >= 2;
    if (encode_tmap_2d(&maps.m[i / 2][i % 2], CU_TENSOR_MAP_DATA_TYPE_UINT8, down ? a.down : a.up,
                       (down ? p.down : p.up).blocks * 16, down ? a.E * a.H : 2 * a.E * a.I,
                       down ? a.ldd : a.ldu, 128, i % 2 ? 32 : 128,
                       CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  constexpr int kSmem = 227 * 1024 - static_cast<int>(sizeof(Routing)) - 512;
  p.stage_kb = (kSmem - 1024 - RING_BYTES) / 1024;
  // A CTA's run touches at most ceil(rows / CTAs) + 1 rows of items (an expert's
  // part of K each), of at most T pairs each; on 152 or 148 SMs that is never more
  // than 264 segments, reached by 64 tokens x 8 of 512 experts at K above 15360.
  for (const MoeProduct* m : {&p.up, &p.down})
    for (int parts = 1; parts <= p.max_parts && parts <= m->stages; ++parts) {
      const int fit = columns_that_fit(p.stage_kb, (m->stages + parts - 1) / parts);
      const int rows = ((p.E < p.T * p.top ? p.E : p.T * p.top) * parts + ctl.sm_count - 1) /
                           ctl.sm_count + 1;
      if (rows * (fit > 1 ? (p.T + fit - 1) / fit : 1) > MAX_SEGMENTS)
        return cudaErrorNotSupported;
    }
  cudaError_t e = cudaFuncSetAttribute(moe_mxfp4_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctl.sm_count);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_main_kernel("moe_mxfp4_kernel", ctl.sm_count, p.T * p.top);
  e = cudaLaunchKernelEx(&cfg, moe_mxfp4_kernel, maps, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mx
}  // namespace mhr
