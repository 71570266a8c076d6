/*
 * mhr_routed.h -- products that go by an index per row, in libmhr_gemm.so: the
 * router of a mixture of experts and its gradient, the sort of its rows by
 * expert, the experts' products with their gradients, and low-rank adapters of
 * many requests.
 *
 * Pointers, streams, errors and threads as in mhr_gemm.h: device pointers on
 * the current device, work enqueued on `stream`, an mhr_status returned,
 * device-side timeouts reported by gemm_check().  Element types are mhr_dtype
 * (mhr_mxfp4.h).  Outputs must not overlap inputs or one another, except where
 * a call says so.  Empty sizes are no-ops.  No call here uses the library's
 * workspace: each can be captured into a graph, and what scratch it needs is
 * the caller's (16-byte aligned; its contents are undefined before and after).
 *
 * What indices on the device hold is not known to the host: an index outside
 * its range never causes an access; each call says what it does instead.
 */
#ifndef MHR_ROUTED_H
#define MHR_ROUTED_H

#include <stdint.h>

#include "mhr_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A router's scores of one token's logits: over all experts, or each by itself. */
typedef enum mhr_score { MHR_SOFTMAX = 0, MHR_SIGMOID = 1 } mhr_score;
/* A group's worth: its best key, or the sum of its two best. */
typedef enum mhr_group_score { MHR_GROUP_MAX = 0, MHR_GROUP_TOP2 = 1 } mhr_group_score;

/*
 * Choose `top` of E experts for each of T tokens.  logits: T x E, pitch ld, of
 * type dtype.  For each token
 *   s     = softmax or sigmoid of its logits;
 *   key   = s + bias (bias: E floats), or without one (NULL) the logit itself,
 *           which orders as s does;
 *   with groups > 1 (E / groups neighbours each): the group_top best groups by
 *           group_score stay (without a bias MHR_GROUP_TOP2 sums two s);
 *   experts = the top largest keys in descending order;
 *   weights = s of the chosen, divided by their sum if `renormalize`, times scale.
 * Ties go to the lowest index and NaN counts as largest, for groups as well.
 * Keys of scores are compared as in 64 bits: where neighbours are too near for
 * 32 the token is done again in double.  A token whose logits are all -inf has
 * scores of zero; a sum of zero leaves weights of zero.  Renormalised weights
 * are taken from the chosen logits alone, so that far below zero they do not
 * underflow together.
 * experts, weights: T x top, contiguous.
 * Limits: E <= 512, top <= 16, groups <= 32 and a divisor of E, top <=
 * group_top * E / groups.
 */
int gemm_routed_choose(int dtype, const void* logits, int64_t T, int64_t E, int64_t ld, int score,
                       const float* bias, int64_t groups, int64_t group_top, int group_score,
                       int64_t top, int renormalize, float scale, int32_t* experts,
                       float* weights, void* stream);

/*
 * The gradient of the logits for one of the weights (grad_weights: T x top
 * floats, contiguous), the choice held fixed; neither it nor the bias has one.
 * grad_logits: T x E, pitch ldg, of type dtype; every element is written.
 * With p the weights over scale:
 *   softmax, renormalised   dl_j = scale p_j (g_j - sum p g) at the chosen, else 0
 *   softmax                 dl_e = scale s_e (g_e [e chosen] - sum p g)
 *   sigmoid, renormalised   dl_j = scale p_j (1 - s_j) (g_j - sum p g)
 *   sigmoid                 dl_j = scale g_j s_j (1 - s_j)
 * An entry of experts outside 0 .. E-1 takes no part; one expert twice in a row
 * adds up.  Scores of zero (see above) have gradients of zero.
 */
int gemm_routed_choose_grad(int dtype, const void* logits, int64_t ld, const int32_t* experts,
                            const float* grad_weights, int64_t T, int64_t E, int64_t top,
                            int score, int renormalize, float scale, void* grad_logits,
                            int64_t ldg, void* stream);

/*
 * The stable order of n entries by expert: order (n) lists the positions of
 * those of expert 0, then of expert 1, and so on, each expert's in ascending
 * order, and last those outside 0 .. E-1; offsets (E + 1) says where each
 * expert's part starts, offsets[E] where the last one ends.  E <= 1024,
 * n < 2^31.
 */
int gemm_routed_sort(const int32_t* experts, int64_t n, int64_t E, int32_t* offsets,
                     int32_t* order, void* stream);

/*
 * The experts' products.  For expert e and each sorted position q, offsets[e]
 * <= q < offsets[e + 1]:
 *   out[scatter ? scatter[q] : q] = x[gather ? gather[q] / top : q] W_e,
 * W_e the K x N matrix at w + e * stride_w, pitch ldw; transposed != 0: W_e^T
 * of the N x K matrix there (the gradient of x: the forward product's weights
 * and the gradient of its output; scatter and gather change places).
 * x: x_rows x K, pitch ldx; out: out_rows x N, pitch ldo; `rows` sorted
 * positions, which is also x_rows without gather and out_rows without scatter.
 * dtype, of x and w: MHR_BF16 or MHR_F16; out_dtype: any.  Sums are held in
 * fp32 on the tensor cores (tcgen05.mma kind::f16), which add by truncation (fp32
 * results go on rounded to nearest every 384 terms), and rounded once.
 *
 * gather and scatter (or NULL): `rows` entries each, as gemm_routed_sort gives
 * them in `order`; `top` divides gather's, so that a (token, slot) pair's row is
 * its token's.  A row of x outside 0 .. x_rows-1 counts as zeros, one of out
 * outside 0 .. out_rows-1 is not written; entries of scatter are distinct.
 * Rows of out of no sorted position, and those at offsets[E] and after, stay as
 * they were.  Offsets below 0 or past `rows` count as that; an expert whose end lies
 * below its start has no positions, and one that starts below an earlier expert's
 * end starts there, so that no position is two experts'.
 * K == 0 writes zeros.  E <= 1024.
 *
 * scratch: gemm_routed_product_scratch bytes, for x's rows in the order of gather
 * (more than 256 of them), and for an x or w whose address, pitch or stride is no
 * multiple of 16 bytes (of w, the experts that have rows); -1: none fits the
 * address space.
 */
int64_t gemm_routed_product_scratch(const void* x, int64_t x_rows, int64_t ldx, int gathered,
                                    const void* w, int64_t ldw, int64_t stride_w, int transposed,
                                    int64_t E, int64_t rows, int64_t K, int64_t N);
int gemm_routed_product(int dtype, const void* x, int64_t x_rows, int64_t ldx,
                        const int32_t* gather, int64_t top, const void* w, int64_t ldw,
                        int64_t stride_w, int transposed, const int32_t* offsets, int64_t E,
                        int out_dtype, void* out, int64_t out_rows, int64_t ldo,
                        const int32_t* scatter, int64_t rows, int64_t K, int64_t N,
                        void* scratch, int64_t scratch_bytes, void* stream);

/*
 * The gradient of the weights of gemm_routed_product: for each expert
 *   out_e = sum over q, offsets[e] <= q < offsets[e + 1], of
 *           x[gather ? gather[q] / top : q]^T grad[scatter ? scatter[q] : q],
 * K x N at out + e * stride_o, pitch ldo; zeros for an expert without rows.
 * grad: grad_rows x N, pitch ldg, of x's type; the rest, and rows outside x or
 * grad, as above.  scratch: gemm_routed_weight_grad_scratch bytes, for rows in the
 * order of gather and of scatter, and for operands as above.
 */
int64_t gemm_routed_weight_grad_scratch(const void* x, int64_t x_rows, int64_t ldx, int gathered,
                                        const void* grad, int64_t grad_rows, int64_t ldg,
                                        int scattered, int64_t rows, int64_t K, int64_t N);
int gemm_routed_weight_grad(int dtype, const void* x, int64_t x_rows, int64_t ldx,
                            const int32_t* gather, int64_t top, const void* grad,
                            int64_t grad_rows, int64_t ldg, const int32_t* scatter,
                            const int32_t* offsets, int64_t E, int out_dtype, void* out,
                            int64_t ldo, int64_t stride_o, int64_t rows, int64_t K, int64_t N,
                            void* scratch, int64_t scratch_bytes, void* stream);

/*
 * Low-rank adapters of many requests, added to a shared projection's result:
 *   out_t = y_t + scales[a] (x_t down_a^T) up_a,  a = which[t], t < T.
 * x: T x K, pitch ldx; down_a: rank x K at down + a * stride_d, pitch ldd; up_a:
 * rank x N at up + a * stride_u, pitch ldu, all of type dtype (MHR_BF16 or
 * MHR_F16); scales: L floats, or NULL for 1; y, out: T x N, of type out_dtype
 * (any).  out may be y itself (the same address and pitch).  A row whose which
 * lies outside 0 .. L-1 has no adapter: out_t = y_t.  Both sums are held in fp32;
 * x_t down_a^T is kept to 2^-22 of the row's largest sum between them, whatever T
 * and the types are; out is rounded once.
 * Infinities and NaN of x, down, y and scales give what the sums above give, and in
 * no other row; an infinity in up gives elements that are not finite, each an
 * infinity or NaN.
 * Limits: L <= 1024, rank <= 128.
 *
 * scratch: gemm_routed_adapters_scratch bytes (0 for few rows; -1 for arguments
 * that the call refuses).
 */
int64_t gemm_routed_adapters_scratch(int dtype, const void* x, int64_t ldx, const void* down,
                                     int64_t ldd, int64_t stride_d, const void* up, int64_t ldu,
                                     int64_t stride_u, int64_t L, int64_t rank, int out_dtype,
                                     int64_t T, int64_t K, int64_t N);
int gemm_routed_adapters(int dtype, const void* x, int64_t ldx, const void* down, int64_t ldd,
                         int64_t stride_d, const void* up, int64_t ldu, int64_t stride_u,
                         const int32_t* which, const float* scales, int64_t L, int64_t rank,
                         int out_dtype, const void* y, int64_t ldy, void* out, int64_t ldo,
                         int64_t T, int64_t K, int64_t N, void* scratch, int64_t scratch_bytes,
                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MHR_ROUTED_H */
