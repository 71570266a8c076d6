/*
 * mhr_mxfp4.h -- microscaled 4-bit floats (MXFP4) in libmhr_gemm.so:
 * quantisation, products, and a mixture-of-experts layer for a few tokens.
 *
 * The format.  A value is an e2m1 code -- 0, 0.5, 1, 1.5, 2, 3, 4 or 6 and a
 * sign in bit 3 -- times an e8m0 scale 2^(code - 127) that 32 consecutive
 * values of a row share (code 255: NaN).  A rows x cols matrix is two arrays:
 *   data    row r starts at r * ld bytes and holds 16 * ceil(cols / 32) bytes,
 *           two codes a byte, the even column in the low half; the last
 *           block's columns past cols hold zero codes.  16-byte aligned, ld a
 *           multiple of 16.
 *   scales  tiles of 128 rows x 4 blocks, 512 bytes each, row-major over
 *           ceil(rows / 128) x ceil(blocks / 4) tiles; the scale of row r and
 *           block b (columns 32 b to 32 b + 31) is byte
 *           (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4 of tile
 *           (r / 128, b / 4).  Bytes past the last row or block are no code of
 *           any value; those past the last block must not be 255.
 *           16-byte aligned, gemm_mxfp4_scale_bytes(rows, cols) bytes.
 *
 * Pointers, streams, errors and threads as in mhr_gemm.h: device pointers on
 * the current device, work enqueued on `stream`, an mhr_status returned,
 * device-side timeouts reported by gemm_check().  Empty sizes are no-ops.
 * gemm_mxfp4_quantize and gemm_mxfp4 can be captured into a graph, and so can a
 * gemm_mxfp4_quantized with M <= 32, K <= 4096 and M ceil(K / 256) <= 50, which
 * quantises inside the product's kernel at any N.  Others may use the library's
 * workspace, which no graph may hold, and return MHR_ERR_CUDA in a capture (which
 * goes on); their C comes, bit for bit, from gemm_mxfp4_quantize and gemm_mxfp4
 * with buffers of the caller's.  gemm_mxfp4_moe always uses the workspace.
 */
#ifndef MHR_MXFP4_H
#define MHR_MXFP4_H

#include <stdint.h>

#include "mhr_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of plain matrices. */
typedef enum mhr_dtype { MHR_F32 = 0, MHR_BF16 = 1, MHR_F16 = 2 } mhr_dtype;

/* Size of the scales of a rows x cols matrix; -1 for a negative size. */
int64_t gemm_mxfp4_scale_bytes(int64_t rows, int64_t cols);

/*
 * Quantise X (rows x cols, row-major, pitch ldx elements, type dtype).
 * transpose == 0: blocks run along X's rows; the packed matrix is X, rows x
 * cols.  transpose != 0: blocks run down X's columns; the packed matrix is
 * X^T, cols x rows -- the form in which gemm_mxfp4 takes its right operand.
 *
 * A block's scale is 2^(floor(log2 m) - 2), m its largest magnitude, and no
 * less than 2^-127; its codes are x / scale rounded to nearest, ties to the
 * even code, magnitudes above 6 to 6.  A block that holds an infinity or a NaN
 * gets the scale NaN and zero codes.  Padding rows and blocks of the scales
 * are written as zero.
 *
 * values (or NULL): also writes what the codes stand for, in X's type and
 * shape with pitch ldv -- exact, since every such value is representable.
 * data, scales and values must not overlap X or one another.
 */
int gemm_mxfp4_quantize(int dtype, const void* X, int64_t rows, int64_t cols, int64_t ldx,
                        int transpose, uint8_t* data, int64_t ldd, uint8_t* scales, void* values,
                        int64_t ldv, void* stream);

/*
 * C = A B: A is M x K in 4 bits, B is given as B^T, N x K in 4 bits (lda, ldb:
 * bytes a row), C is M x N, row-major, pitch ldc elements, type c_dtype.
 * Products are exact, sums are held in fp32 on the tensor cores
 * (tcgen05.mma kind::mxf4, block scales applied there), C is rounded once.
 * K == 0 writes zeros.  C must not overlap an operand.
 */
int gemm_mxfp4(int c_dtype, const uint8_t* A, const uint8_t* A_scales, const uint8_t* Bt,
               const uint8_t* Bt_scales, void* C, int64_t M, int64_t N, int64_t K, int64_t lda,
               int64_t ldb, int64_t ldc, void* stream);

/*
 * The same with A (M x K, row-major, pitch lda elements, type a_dtype)
 * quantised on the way as gemm_mxfp4_quantize does along its rows: the C of
 * quantising and then multiplying, bit for bit.  Few rows are quantised inside
 * the product's kernel; the packed A of more lives in the library's workspace
 * (see mhr_gemm.h).
 */
int gemm_mxfp4_quantized(int a_dtype, const void* A, int c_dtype, const uint8_t* Bt,
                         const uint8_t* Bt_scales, void* C, int64_t M, int64_t N, int64_t K,
                         int64_t lda, int64_t ldb, int64_t ldc, void* stream);

/*
 * A mixture-of-experts layer for a few tokens, in one kernel.  x: T x H bf16;
 * router: E x H bf16; up: a packed 2 E I x H matrix, expert e's gate rows from
 * row 2 e I and its up rows from row (2 e + 1) I; down: a packed E H x I
 * matrix, expert e's rows from row e H; y: T x H bf16; experts, weights:
 * T x top, contiguous.  For each token t:
 *   logits = router x_t (fp32), experts = the top largest in descending order
 *   (ties to the lowest index, a NaN counts as largest), weights = their
 *   softmax (over the chosen ones: the full softmax renormalised);
 *   y_t = sum over the chosen of weight * down_e (silu(gate_e x_t) * (up_e x_t)),
 * rounded once to bf16; sums are fp32.  For the tensor cores x and the inner
 * vector are written as sums of eight 4-bit values a block of 32, which leaves
 * less than 2^-22 of the block's largest magnitude, or 2^-129 where that is
 * more (blocks below some 2^-107).
 * A token whose x holds an infinity or a NaN has weights of NaN, as the softmax
 * of such logits, and a y of NaN.  So has one with an inner value that is not
 * finite (a product past fp32's range; the sum above could be an infinity).
 * Limits: T <= 64, top <= 16, E <= 512, H and I <= 16384.
 * The call needs every SM at once (a cooperative launch): it waits for kernels
 * before it on the device to leave.
 */
int gemm_mxfp4_moe(const uint16_t* x, int64_t ldx, const uint16_t* router, int64_t ldr,
                   const uint8_t* up, const uint8_t* up_scales, int64_t ldu, const uint8_t* down,
                   const uint8_t* down_scales, int64_t ldd, uint16_t* y, int64_t ldy,
                   int32_t* experts, float* weights, int64_t T, int64_t E, int64_t top, int64_t H,
                   int64_t I, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MHR_MXFP4_H */
