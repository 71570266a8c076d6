// Microscaled 4-bit floats (MXFP4): the packed format, its element arithmetic,
// and the tcgen05 instructions that multiply it.
//
// A value is an e2m1 code (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1,
// 1.5, 2, 3, 4, 6) times an e8m0 scale 2^(code - 127) shared by 32
// consecutive values of a row.  A rows x cols matrix is
//   data    row r at r * ld bytes, ld a multiple of 16, two codes a byte, the
//           even column in the low half; a row's last block is padded with
//           zero codes to 32 columns;
//   scales  tiles of 128 rows x 4 blocks, 512 bytes each, in row-major order of
//           tiles: byte (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4 of a tile.
//           This is the order in which one tcgen05.cp.32x128b.warpx4 moves a
//           tile into TMEM for the block-scaled MMA.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "mhr_device.cuh"
#include "mxfp4_internal.h"

namespace mhr {
namespace mx {

// ------------------------------------------------------------------ elements

// Eight floats -> a word of e2m1 codes (nearest, ties to the even code,
// saturating at 6), value i in bits [4 i, 4 i + 4).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The largest magnitude of three; NaN if one is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_abs8(const float (&v)[8]) {
  return max_abs3(max_abs3(max_abs3(v[0], v[1], v[2]), v[3], v[4]),
                  max_abs3(v[5], v[6], v[7]), 0.f);
}

// The codes of eight values over their block's scale.  Two products an instruction,
// as the maximum takes two more values in one: quantising along rows issued 104
// instructions for 8 columns before and was held to 5.4 of the 6.6 TB/s it runs at.
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], float inv) {
  float y[8];
  uint64_t ii;
  asm("mov.b64 %0, {%1, %1};" : "=l"(ii) : "f"(inv));
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%2, %3};\n\tmul.rn.f32x2 t, t, %4;\n\t"
        "mov.b64 {%0, %1}, t;\n\t}"
        : "=f"(y[i]), "=f"(y[i + 1])
        : "f"(x[i]), "f"(x[i + 1]), "l"(ii));
  return e2m1x8(y);
}

// Byte `I` of a word of e2m1 codes -> its two values as f16x2 (exact).
template <int I>
__device__ __forceinline__ uint32_t e2m1_to_f16x2(uint32_t codes) {
  uint32_t r;
  if constexpr (I == 0)
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}" : "=r"(r) : "r"(codes));
  else if constexpr (I == 1)
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b1;\n\t}" : "=r"(r) : "r"(codes));
  else if constexpr (I == 2)
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b2;\n\t}" : "=r"(r) : "r"(codes));
  else
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b3;\n\t}" : "=r"(r) : "r"(codes));
  return r;
}

// The scale of a block whose largest magnitude has the fp32 bits `amax` (sign
// cleared): 2^(floor(log2 amax) - 2), so that the largest value lies in [4, 8)
// (above 6 it saturates), no less than 2^-127; 255 (NaN) for a block that
// holds an infinity or a NaN.  On the bits: fp32's exponent field is
// floor(log2) + 127 (0 below 2^-126, where the lower limit applies anyway).
__device__ __forceinline__ uint32_t scale_code(uint32_t amax) {
  const uint32_t e = amax >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 1 / scale: 2^(127 - code).  Exact and normal for codes 0 to 252, all that
// scale_code gives but NaN, whose blocks get zero codes.
__device__ __forceinline__ float scale_inverse(uint32_t code) {
  return code == 255u ? 0.f : __uint_as_float((254u - code) << 23);
}
// The scale itself, 2^(code - 127): code 0 is the subnormal 2^-127.
__device__ __forceinline__ float scale_value(uint32_t code) {
  return code == 255u ? __uint_as_float(0x7fffffffu)
                      : __uint_as_float(code ? code << 23 : 1u << 22);
}

// Byte offset of the scale of (row, block) in the tiled array, kt tiles a row.
__host__ __device__ __forceinline__ int64_t scale_offset(int64_t row, int64_t block, int64_t kt) {
  return ((row >> 7) * kt + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
         (block & 3);
}

// ------------------------------------------------------------------ values

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// ------------------------------------------------------------------ tcgen05

// Instruction descriptor of kind::mxf4, dense, K = 64, fp32 accumulator: B's
// scale id in [4,6), A and B formats in [7,10) and [10,13) (1 = e2m1), N >> 3
// in [17,23), scale type in bit 23 (1 = e8m0), M >> 7 in [27,29), A's scale id
// in [29,31).  Both operands are K-major.  A scale id of 0 or 2 picks the first
// or second pair of the 4 scales that a TMEM word holds for a row.
__host__ __device__ constexpr uint32_t make_idesc_mxf4(uint32_t m, uint32_t n, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (1u << 23) |
         ((m >> 7) << 27) | (sf_id << 29);
}

// The issuing warp runs its loop converged, so that addresses and descriptors
// stay in uniform registers, and one elected lane issues: with the loop inside
// an `if (lane == 0)`, each MMA cost some 114 cycles to issue (GB300), nearly
// the 128 that it takes.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Low word of a shared-memory descriptor: the address in 16-byte units and,
// for operands, the K-major leading offset (unused by swizzled layouts, 1).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | (1u << 16);
}
// High words: 128-byte swizzle with 1024 bytes between groups of 8 rows
// (operands); no swizzle with 128 bytes between them (scale tiles).
constexpr uint32_t DESC_HI_SW128 = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t DESC_HI_SCALES = (128u >> 4) | (1u << 14);

// D (+)= (A * scales) (B * scales) over 64 columns of K: two blocks of 32 a
// row, the scales in TMEM.
template <int GROUP>
__device__ __forceinline__ void mma_mxf4(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                         uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                         uint32_t accumulate) {
  if constexpr (GROUP == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X"
        " [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate),
        "r"(DESC_HI_SW128)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X"
        " [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate),
        "r"(DESC_HI_SW128)
        : "memory");
}

// One scale tile (128 rows x 4 blocks, 512 bytes of shared memory) into 4 TMEM
// columns: row r's four scales in column r / 32 of lane r % 32, repeated in
// each of the four lane quarters.  Unswizzled: 32 rows of 16 bytes, 8 rows
// (128 bytes) a group.  GROUP 2 copies in both CTAs, each from its own shared
// memory at the same offset.
template <int GROUP>
__device__ __forceinline__ void copy_scale_tile(uint32_t d_tmem, uint32_t s_lo) {
  if constexpr (GROUP == 1)
    asm volatile(
        "{\n\t.reg .b64 s;\n\tmov.b64 s, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], s;\n\t}" ::"r"(d_tmem),
        "r"(s_lo), "r"(DESC_HI_SCALES)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .b64 s;\n\tmov.b64 s, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], s;\n\t}" ::"r"(d_tmem),
        "r"(s_lo), "r"(DESC_HI_SCALES)
        : "memory");
}

// Untiled bulk copy: both addresses and the size multiples of 16 bytes.
// `bar` may be a barrier of the pair's other CTA (a shared::cluster address).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// 3-D tiled load into this CTA's shared memory; the bytes complete on the
// mbarrier at `bar_cluster`, which may be in the peer CTA of the pair.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int32_t x, int32_t y,
                                                 int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 8 consecutive fp32 columns of one TMEM lane per thread (32x32b, x8).
__device__ __forceinline__ void tmem_ld_8cols(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

}  // namespace mx
}  // namespace mhr
