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
// registers that the weights are unpacked into.  A warp walks K in steps of
// 128 columns, four blocks of 32; lane 4 g + q loads the 16 bytes of block q
// of rows g and g + 8 straight from global memory, four steps ahead.  The
// sum over k does not mind an order, so lane q's k indices are its own block's
// and an operand needs no shuffle; the columns side is laid out in shared
// memory in that order.  e2m1 is exact in f16, and so is its product with the
// block's scale relative to the largest of the four (a power of two not above
// 1; below 2^-24 of the row's largest block it vanishes, which is below fp32's
// rounding of the sum).  The largest scale multiplies the fp32 sum of the step.
//
// Columns in f16: x in bf16 (8 significant bits) and h in fp32 are scaled by a
// power of two per token or pair that puts the largest magnitude in [2^12,
// 2^13), so that values down to 2^-26 of the largest keep f16's 11 bits.  x
// stays exact but for values below 2^-29 of its largest.  h is rounded to 11
// bits, an eighth of the final rounding to bf16.
//
// The partial outputs of a pair go to the workspace; the group of warps that
// finishes the last expert of 16 rows adds a token's pairs in their order and
// rounds: results do not depend on the schedule.
#include "mhr_gemm.h"
#include "mhr_mxfp4.h"
#include "mxfp4_common.cuh"

namespace mhr {
namespace mx {
namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int DEPTH = 4;                       // steps of 128 columns a warp has in flight
constexpr int MAX_PAIRS = MOE_MAX_TOKENS * MOE_MAX_TOP;
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
  uint32_t* control;       // [0] barrier arrivals, [1] exits, [2 ..] finished experts of 16 rows
  int32_t row_tiles;       // ceil(H / 16)
  int32_t stage_bytes;     // shared memory for staged columns
  uint32_t* status;
  uint64_t wait_limit_ns;
  int32_t inject_stall;
};

struct Routing {  // shared memory
  int32_t expert[MAX_PAIRS];          // of pair t * top + k
  float weight[MAX_PAIRS];
  int32_t list[MAX_PAIRS];            // pairs, expert by expert
  int32_t count[MOE_MAX_EXPERTS];     // pairs of an expert
  int32_t offset[MOE_MAX_EXPERTS];    // its first place in list
  int32_t active[MOE_MAX_EXPERTS];    // the experts that some pair has
  int32_t num_active;
  int32_t fill[MOE_MAX_EXPERTS];
  int32_t last;                       // (by group) whether this was a tile's last expert
  int32_t abort;
};

__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void mma_f16_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1,
                                                uint32_t a2, uint32_t a3, uint32_t b0,
                                                uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The largest of four scale codes, and 2^(code q - largest) as f16x2.
__device__ __forceinline__ uint32_t step_scale(uint32_t codes, int q, uint32_t& largest) {
  const uint32_t m = max(max(codes & 255u, (codes >> 8) & 255u),
                         max((codes >> 16) & 255u, codes >> 24));
  largest = m;
  const uint32_t d = min(m - ((codes >> (8 * q)) & 255u), 126u);
  const __half h = __float2half_rn(__uint_as_float((127u - d) << 23));
  const uint32_t b = __half_as_ushort(h);
  return b | (b << 16);
}

// The power of two that puts a magnitude with these fp32 bits in [2^12, 2^13);
// 1 for zero, infinities and NaNs (which f16 keeps).
__device__ __forceinline__ float f16_multiplier(uint32_t amax) {
  const int e = static_cast<int>(amax >> 23);
  if (amax == 0 || e == 255) return 1.f;
  const int m = 127 + 12 - (e - 127);  // biased exponent of the multiplier
  return __uint_as_float(static_cast<uint32_t>(min(max(m, 1), 254)) << 23);
}

__device__ __forceinline__ void load8_bf16(const __nv_bfloat16* p, int left, bool vec,
                                           float (&v)[8]) {
  if (vec && left >= 8) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? __bfloat162float(p[i]) : 0.f;
  }
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

// Step 1, all warps of the grid: router logits (a warp takes one expert and
// four tokens), each token's f16 multiplier, and zeroed pair maxima.
__device__ void route_logits(const MoeParams& p) {
  const int lane = threadIdx.x & 31;
  const int warp = (threadIdx.x >> 5) * gridDim.x + blockIdx.x;  // neighbours on other SMs
  const int warps = gridDim.x * WARPS;
  const bool vx = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ldx % 8 == 0;
  const bool vr = reinterpret_cast<uintptr_t>(p.router) % 16 == 0 && p.ldr % 8 == 0;
  const int quads = (p.T + 3) / 4;
  for (int task = warp; task < p.E * quads; task += warps) {
    const int e = task / quads, t0 = (task - e * quads) * 4;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int k = lane * 8; k < p.H; k += 256) {
      float w[8];
      load8_bf16(p.router + e * p.ldr + k, p.H - k, vr, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (t0 + j < p.T) {
          float v[8];
          load8_bf16(p.x + (t0 + j) * p.ldx + k, p.H - k, vx, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[j] = fmaf(w[i], v[i], sum[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int d = 16; d; d >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], d);
      if (lane == 0 && t0 + j < p.T) p.logits[(t0 + j) * p.E + e] = sum[j];
    }
  }
  for (int t = warps - 1 - warp; t < p.T; t += warps) {  // from the warps with no logits left
    uint32_t amax = 0;
    for (int k = lane * 8; k < p.H; k += 256) {
      float v[8];
      load8_bf16(p.x + t * p.ldx + k, p.H - k, vx, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    if (lane == 0) p.x_mult[t] = f16_multiplier(amax);
    if (lane < p.top) p.h_max[t * p.top + lane] = 0;
  }
}

// Step 2, in every CTA alike: the top experts of each token, ties to the lowest
// index, their weights, and the pairs sorted by expert.
__device__ void route_choose(const MoeParams& p, Routing& r) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int PER_LANE = MOE_MAX_EXPERTS / 32;
  for (int t = warp; t < p.T; t += WARPS) {
    // keys that order as (logit, then lowest expert); a NaN counts as largest
    uint64_t key[PER_LANE];
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) {
      const int e = lane + 32 * i;
      key[i] = 0;
      if (e < p.E) {
        float v = __ldcg(p.logits + t * p.E + e);
        if (v == 0.f) v = 0.f;  // -0 and 0 tie
        const uint32_t b = __float_as_uint(v);
        const uint32_t o = v != v ? 0xffffffffu : (b >> 31 ? ~b : b | 0x80000000u);
        key[i] = (static_cast<uint64_t>(o) << 32) | (0xffffffffu - e);
      }
    }
    float chosen = 0.f, first = 0.f;
    for (int k = 0; k < p.top; ++k) {
      uint64_t best = 0;
#pragma unroll
      for (int i = 0; i < PER_LANE; ++i) best = key[i] > best ? key[i] : best;
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, best, d);
        best = o > best ? o : best;
      }
#pragma unroll
      for (int i = 0; i < PER_LANE; ++i)
        if (key[i] == best) key[i] = 0;
      const int e = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
      const float logit = __ldcg(p.logits + t * p.E + e);
      if (k == 0) first = logit;
      if (lane == k) {
        chosen = logit;
        r.expert[t * p.top + k] = e;
      }
    }
    const float w = lane < p.top ? expf(chosen - first) : 0.f;
    float sum = w;
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane < p.top) r.weight[t * p.top + lane] = w / sum;
  }
  const int pairs = p.T * p.top;
  for (int e = threadIdx.x; e < p.E; e += THREADS) r.count[e] = r.fill[e] = 0;
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
      if (e0 + lane < p.E) r.offset[e0 + lane] = offset + scan - c;
      if (c > 0) r.active[active + __popc(has & ((1u << lane) - 1))] = e0 + lane;
      active += __popc(has);
      offset += __shfl_sync(0xffffffffu, scan, 31);
    }
    if (lane == 0) r.num_active = active;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += THREADS) {
    const int e = r.expert[i];
    // (an expert's pairs in any order: each is a column of its own)
    r.list[r.offset[e] + atomicAdd(&r.fill[e], 1)] = i;
    if (blockIdx.x == 0) {
      p.experts[i] = e;
      p.weights[i] = r.weight[i];
    }
  }
  __syncthreads();
}

// Steps 3 and 4.  UP: units of 8 gate rows and the same 8 up rows, columns x,
// K = H; otherwise units of 16 rows of the down matrix, columns h, K = I.
// The CTA takes an equal run of all units, expert by expert; for each expert
// it stages up to 8 NT of its pairs' columns, and groups of warps take the
// units in turn, each warp an equal part of K.
template <int NT, bool UP>
__device__ void product(const MoeParams& p, Routing& r, uint8_t* staged, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int kt = UP ? p.kt_h : p.kt_i;
  const int blocks = UP ? (p.H + 31) / 32 : (p.I + 31) / 32;
  const int tiles = UP ? (p.I + 7) / 8 : p.row_tiles;
  const int64_t units = static_cast<int64_t>(r.num_active) * tiles;
  const int64_t u_begin = units * blockIdx.x / gridDim.x;
  const int64_t u_end = units * (blockIdx.x + 1) / gridDim.x;
  const uint8_t* data = UP ? p.up : p.down;
  const uint8_t* scales = UP ? p.up_s : p.down_s;
  const int64_t ld = UP ? p.ldu : p.ldd;
  const int pitch = kt * 256 + 64;  // 64 past a multiple of 128: neighbouring rows' banks differ
  const int capacity = min(8 * NT, p.stage_bytes / pitch);
  // warps a unit: as many units at once as the CTA has, down to one warp each
  int ws = WARPS;
  while (ws > 1 && (WARPS / ws < u_end - u_begin || ws > kt)) ws >>= 1;
  ws = max(ws, WARPS / 8);  // (named barriers 1 to 8)
  const int groups = WARPS / ws, group = warp / ws, part = warp - group * ws;
  const int k_begin = kt * part / ws, k_end = kt * (part + 1) / ws;
  const bool vx = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ldx % 8 == 0;

  for (int64_t seg = u_begin; seg < u_end;) {
    const int ai = static_cast<int>(seg / tiles), e = r.active[ai];
    const int t_begin = static_cast<int>(seg - static_cast<int64_t>(ai) * tiles);
    const int t_end = static_cast<int>(min(static_cast<int64_t>(tiles), t_begin + u_end - seg));
    for (int c0 = 0; c0 < r.count[e]; c0 += capacity) {
      const int cols = min(capacity, r.count[e] - c0);
      const int32_t* list = r.list + r.offset[e] + c0;
      __syncthreads();  // the staged columns before these have been read
      for (int i = threadIdx.x; i < cols * kt * 16; i += THREADS) {
        const int c = i / (kt * 16), piece = i - c * (kt * 16), k = piece * 8;
        float v[8];
        float mult;
        if (UP) {
          const int t = list[c] / p.top;
          mult = __ldcg(p.x_mult + t);
          if (k < p.H)
            load8_bf16(p.x + t * p.ldx + k, p.H - k, vx, v);
          else
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.f;
        } else {
          mult = f16_multiplier(__ldcg(p.h_max + list[c]));
          const float4* src = reinterpret_cast<const float4*>(
              p.h + static_cast<int64_t>(list[c]) * p.kt_i * 128 + k);
          const float4 a = __ldcg(src), b = __ldcg(src + 1);
          const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = k + j < p.I ? f[j] : 0.f;
        }
        // piece 4 q + c of a step at place 4 c + q: a load of the four lanes
        // of a row is then 64 contiguous bytes
        const int step = piece >> 4, at = piece & 15;
        *reinterpret_cast<uint4*>(staged + c * pitch + step * 256 +
                                  ((at & 3) * 4 + (at >> 2)) * 16) = to_f16x8(v, mult);
      }
      __syncthreads();
      const int ntiles = (cols + 7) / 8;

      // the warp's walk: units t_begin + group, + groups, ...; steps k_begin to k_end of each
      struct Slot {
        uint4 a, b;
        uint32_t sa, sb;
      } slot[DEPTH];
      int lt = t_begin + group, lk = k_begin;
      const uint8_t *pa, *pb, *psa, *psb;
      auto rows_of = [&](int tile) {
        int64_t ra, rb;
        if (UP) {
          ra = static_cast<int64_t>(e) * 2 * p.I + min(tile * 8 + g, p.I - 1);
          rb = ra + p.I;
        } else {
          ra = static_cast<int64_t>(e) * p.H + min(tile * 16 + g, p.H - 1);
          rb = static_cast<int64_t>(e) * p.H + min(tile * 16 + 8 + g, p.H - 1);
        }
        pa = data + ra * ld + q * 16;
        pb = data + rb * ld + q * 16;
        psa = scales + scale_offset(ra, 0, kt);
        psb = scales + scale_offset(rb, 0, kt);
      };
      auto load = [&](Slot& s) {
        if (lt >= t_end) return;
        if (lk * 4 + q < blocks) {
          s.a = ldg_stream(pa + lk * 64);
          s.b = ldg_stream(pb + lk * 64);
        } else {
          s.a = s.b = make_uint4(0, 0, 0, 0);
        }
        s.sa = __ldg(reinterpret_cast<const uint32_t*>(psa + static_cast<int64_t>(lk) * 512));
        s.sb = __ldg(reinterpret_cast<const uint32_t*>(psb + static_cast<int64_t>(lk) * 512));
        if (++lk == k_end) {
          lk = k_begin;
          lt += groups;
          if (lt < t_end) rows_of(lt);
        }
      };
      float acc[NT][4];
      auto clear = [&] {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
      };
      auto step = [&](const Slot& s, int k) {
        uint32_t la, lb;
        const uint32_t ma = step_scale(s.sa, q, la), mb = step_scale(s.sb, q, lb);
        float sum[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[n][i] = 0.f;
        const uint32_t wa[4] = {s.a.x, s.a.y, s.a.z, s.a.w};
        const uint32_t wb[4] = {s.b.x, s.b.y, s.b.z, s.b.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t a0 = hmul2(e2m1_to_f16x2<0>(wa[c]), ma);
          const uint32_t a1 = hmul2(e2m1_to_f16x2<1>(wa[c]), ma);
          const uint32_t a2 = hmul2(e2m1_to_f16x2<2>(wa[c]), ma);
          const uint32_t a3 = hmul2(e2m1_to_f16x2<3>(wa[c]), ma);
          const uint32_t b0 = hmul2(e2m1_to_f16x2<0>(wb[c]), mb);
          const uint32_t b1 = hmul2(e2m1_to_f16x2<1>(wb[c]), mb);
          const uint32_t b2 = hmul2(e2m1_to_f16x2<2>(wb[c]), mb);
          const uint32_t b3 = hmul2(e2m1_to_f16x2<3>(wb[c]), mb);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (n < ntiles) {
              const int col = min(n * 8 + g, cols - 1);
              const uint4 x = *reinterpret_cast<const uint4*>(staged + col * pitch + k * 256 +
                                                              c * 64 + q * 16);
              mma_f16_16x8x16(sum[n], a0, b0, a1, b1, x.x, x.y);
              mma_f16_16x8x16(sum[n], a2, b2, a3, b3, x.z, x.w);
            }
          }
        }
        const float fa = scale_value(la), fb = scale_value(lb);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[n][0] = fmaf(sum[n][0], fa, acc[n][0]);
          acc[n][1] = fmaf(sum[n][1], fa, acc[n][1]);
          acc[n][2] = fmaf(sum[n][2], fb, acc[n][2]);
          acc[n][3] = fmaf(sum[n][3], fb, acc[n][3]);
        }
      };
      uint32_t turn = 0;
      // A finished unit: the group's parts of K meet in shared memory (two
      // buffers in turn, so one barrier a unit) and are added in their order.
      auto finish = [&](int tile) {
        float* buf = red + (turn & 1) * (WARPS * NT * 128);
        ++turn;
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (n < ntiles)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              buf[warp * (NT * 128) + (n * 4 + i) * 32 + lane] = acc[n][i];
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(ws * 32) : "memory");
        const float* mine = buf + group * ws * (NT * 128);
        if (UP) {
          // 64 outputs of a column tile: (i, lane) -> row lane / 4, column 2 (lane % 4) + i
          for (int o = part; o < ntiles * 2; o += ws) {
            const int n = o >> 1, i = o & 1, col = n * 8 + q * 2 + i;
            float gate = 0.f, value = 0.f;
            for (int w = 0; w < ws; ++w) {
              gate += mine[w * (NT * 128) + (n * 4 + i) * 32 + lane];
              value += mine[w * (NT * 128) + (n * 4 + 2 + i) * 32 + lane];
            }
            const int row = tile * 8 + g;
            const bool in = col < cols && row < p.I;
            const int pair = list[min(col, cols - 1)];
            const float back = 1.f / __ldcg(p.x_mult + pair / p.top);  // a power of two
            gate *= back;
            value *= back;
            const float hv = gate / (1.f + expf(-gate)) * value;
            if (in) p.h[static_cast<int64_t>(pair) * p.kt_i * 128 + row] = hv;
            uint32_t m = in ? __float_as_uint(hv) & 0x7fffffffu : 0u;
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
            if (g == 0 && col < cols) atomicMax(p.h_max + pair, m);
          }
        } else {
          // 128 outputs of a column tile: i picks row lane / 4 (+ 8) and the column's parity
          for (int o = part; o < ntiles * 4; o += ws) {
            const int n = o >> 2, i = o & 3, col = n * 8 + q * 2 + (i & 1);
            float v = 0.f;
            for (int w = 0; w < ws; ++w) v += mine[w * (NT * 128) + (n * 4 + i) * 32 + lane];
            const int row = tile * 16 + g + (i >> 1) * 8;
            if (col < cols && row < p.H) {
              const int pair = list[col];
              const float back = 1.f / f16_multiplier(__ldcg(p.h_max + pair));
              p.part[static_cast<int64_t>(pair) * p.H + row] = v * back * r.weight[pair];
            }
          }
          // the last expert (and the last of its column runs) of these 16
          // rows adds each token's pairs in their order
          if (c0 + cols < r.count[e]) return;
          __threadfence();
          asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(ws * 32) : "memory");
          int done = 0;
          if (part == 0 && lane == 0)
            done = atomicAdd(p.control + 2 + tile, 1u) == static_cast<uint32_t>(r.num_active - 1);
          int* flag = reinterpret_cast<int*>(red + 2 * (WARPS * NT * 128)) + group;
          if (part == 0 && lane == 0) *flag = done;
          asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(ws * 32) : "memory");
          if (*flag) {
            __threadfence();
            for (int o = part * 32 + lane; o < p.T * 16; o += ws * 32) {
              const int t = o >> 4, row = tile * 16 + (o & 15);
              if (row < p.H) {
                float sum = 0.f;
                for (int k = 0; k < p.top; ++k)
                  sum += __ldcg(p.part + static_cast<int64_t>(t * p.top + k) * p.H + row);
                p.y[t * p.ldy + row] = __float2bfloat16_rn(sum);
              }
            }
          }
        }
      };

      if (lt < t_end) rows_of(lt);
      int ct = t_begin + group, ck = k_begin;
      clear();
      if (k_begin == k_end) {  // fewer steps than warps: this one only adds
        for (; ct < t_end; ct += groups) finish(ct);
      } else {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) load(slot[d]);
        while (ct < t_end) {
#pragma unroll
          for (int d = 0; d < DEPTH; ++d) {
            if (ct < t_end) {
              step(slot[d], ck);
              load(slot[d]);
              if (++ck == k_end) {
                finish(ct);
                clear();
                ck = k_begin;
                ct += groups;
              }
            }
          }
        }
      }
    }
    seg += t_end - t_begin;
  }
}

template <int NT>
__global__ void __launch_bounds__(THREADS, 1) moe_mxfp4_kernel(const MoeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                             ~static_cast<uintptr_t>(127));
  __shared__ Routing r;
  uint8_t* staged = smem;
  float* red = reinterpret_cast<float*>(smem + p.stage_bytes);
  if (threadIdx.x == 0) r.abort = 0;
  route_logits(p);
  if (grid_barrier(p, r, 1)) {
    route_choose(p, r);
    product<NT, true>(p, r, staged, red);
    if (grid_barrier(p, r, 2)) product<NT, false>(p, r, staged, red);
  }
  // The last CTA to leave clears the counters for the next call.
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    r.last = atomicAdd(p.control + 1, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (r.last)
    for (int i = threadIdx.x; i < 2 + p.row_tiles; i += THREADS) p.control[i] = 0;
}

template <int NT>
cudaError_t launch_t(MoeParams p, const DeviceCtl& ctl, cudaStream_t s) {
  constexpr int kSmem = 227 * 1024 - static_cast<int>(sizeof(Routing)) - 256;
  constexpr int kRed = 2 * WARPS * NT * 128 * 4 + 64;
  auto kern = moe_mxfp4_kernel<NT>;
  // no more shared memory than the columns need: the rest is L1
  const int pitch = (p.kt_h > p.kt_i ? p.kt_h : p.kt_i) * 256 + 64;
  const int cols = p.T < 8 * NT ? p.T : 8 * NT;
  const int room = (kSmem - 128 - kRed) / 16 * 16;
  if (room < pitch) return cudaErrorInvalidValue;
  p.stage_bytes = static_cast<int64_t>(cols) * pitch < room ? cols * pitch : room;
  const int smem = p.stage_bytes + kRed + 128;
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
  p.row_tiles = static_cast<int32_t>((a.H + 15) / 16);
  p.status = ctl.status;
  p.wait_limit_ns = ctl.wait_limit_ns;
  p.inject_stall = ctl.inject_stall;
  // columns an expert can have are at most T: tiles of 8
  if (a.T <= 8) return launch_t<1>(p, ctl, s);
  if (a.T <= 16) return launch_t<2>(p, ctl, s);
  return launch_t<4>(p, ctl, s);
}

}  // namespace mx
}  // namespace mhr
