/*
 * mpgemm_ops.h -- C ABI of the operators beside the GEMM for gfx950 (AMD
 * Instinct MI355X), in libmpgemm_ops.so: products of 8-bit codes with scales,
 * and products of tokens with experts.
 *
 *   mpgemm_quantize_rows          rows to 8-bit codes with a scale per row
 *   mpgemm_i8_gemm                product of codes with scales per token and
 *                                 channel, one weight matrix or one per expert
 *   mpgemm_route                  (token, slot) pairs sorted by expert
 *   mpgemm_gather_rows            tokens' rows into that order
 *   mpgemm_combine_rows           experts' rows back to tokens, weighted
 *   mpgemm_combine_rows_backward  its gradients
 *   mpgemm_grouped                16-bit products of each expert's rows
 *   mpgemm_grouped_wgrad          their gradient by the weights
 *
 * The rules of mpgemm.h hold here too: device pointers the caller owns, sizes
 * and leading dimensions in elements, work enqueued on `stream` (a
 * hipStream_t of the current device; NULL the default one), nothing
 * allocated, kept or synchronized, 0 or a negative MPGEMM_E* code (argument
 * errors before any HIP call).  Every call may be recorded into a HIP graph.
 * Results are the same from run to run.  Outputs must not overlap inputs or
 * each other.  Any size >= 0 is accepted within the limits named below
 * (MPGEMM_EDIM beyond them), and any element alignment.  A token's row has at
 * most 2^28 values; a product has at most 2^22 tiles, of at least 16x16 values
 * each and of up to 256x256 where the rows are many.
 *
 * Experts.  T tokens with top_k slots each make T*top_k pairs, pair
 * t*top_k + s for slot s of token t.  Sorted by expert they take positions
 * 0 .. R-1 (R = T*top_k); the rows of expert e are positions offsets[e] ..
 * offsets[e+1]-1 (offsets: groups + 1 int32 values in device memory).  Pairs
 * without an expert (an id outside 0 .. experts-1: a dropped pair, an expert
 * of another device) have no position, and rows from offsets[groups] on are
 * neither read nor written.  A group may be empty.  At most
 * MPGEMM_MAX_GROUPS groups.
 *
 * Index arrays (offsets, order, position) are read on the device and cannot
 * be refused: ranges are clamped to the operands and an index outside them
 * counts as absent, so wrong ones give wrong results but no access outside
 * the operands.
 */
#ifndef MPGEMM_OPS_H
#define MPGEMM_OPS_H

#include <stdint.h>

#include "mpgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types (the first two are MPGEMM_IN_F16 and MPGEMM_IN_BF16). */
#define MPGEMM_T_F16 0
#define MPGEMM_T_BF16 1
#define MPGEMM_T_F32 2

/* Types of expert ids. */
#define MPGEMM_ID_I32 0
#define MPGEMM_ID_I64 1

#define MPGEMM_MAX_GROUPS 1024
/* Largest K of mpgemm_i8_gemm: 131071 * 128 * 128 < 2^31, so no sum of
 * products overflows its 32 bits. */
#define MPGEMM_I8_MAX_K 131071

/*
 * Rows to 8-bit codes:  with m = max_h |x[h]|,
 *     scale = m / 127,   code[h] = the whole number nearest to 127*x[h]/m
 * (the exact quotient; the even one in the middle), so x[h] is about
 * code[h] * scale and |code[h]| <= 127.  A row of zeros has scale 0 and codes
 * 0.  A row that holds an infinity or a NaN has a NaN scale and codes 0: it
 * reaches the product as NaN.
 *
 * X: T x H of x_type, ldx >= max(1,H).  Q: R x H codes, ldq >= max(1,H).
 * scale: R floats.  order NULL: row i of Q is row i of X, R == T.  Otherwise
 * row p of Q is row order[p] / top_k of X (R values from mpgemm_route), and
 * rows whose order is outside 0 .. T*top_k-1 keep what they hold.
 * T and R below 2^31, H at most 2^28.  workspace: see mpgemm_rows_workspace.
 */
int mpgemm_quantize_rows(int x_type, int64_t T, int64_t H, const void *X, int64_t ldx,
                         const int32_t *order, int64_t R, int64_t top_k,
                         int8_t *Q, int64_t ldq, float *scale,
                         void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Product of 8-bit codes:
 *     C[i][j] = (sum_k A[i][k] * W[j][k]) * scale_a[i] * scale_w[j] (+ bias[j])
 * The sum is exact; it is rounded to FP32 and multiplied by scale_a[i] in FP32;
 * scale_w[j] and the bias follow in one fused multiply-add in FP32 (without a
 * bias, one product); out_type (MPGEMM_T_*) rounds once more.
 *
 * A: M x K codes, lda >= max(1,K).  W: N x K codes (a column-major K x N
 * matrix: K consecutive), ldw >= max(1,K).  C: M x N, ldc >= max(1,N).
 * scale_a: M floats; scale_w: N; bias: N or NULL.
 *
 * offsets NULL: one product, groups must be 1.  Otherwise rows offsets[g] ..
 * offsets[g+1]-1 of A and C use the weights at W + g*stride_w and row g of
 * scale_w and bias (groups x N, contiguous).
 * K <= MPGEMM_I8_MAX_K; M and N below 2^31; 16 rows of A and of W within 2 GiB
 * (else MPGEMM_ELD).
 */
int mpgemm_i8_gemm(int out_type, int64_t groups, int64_t M, int64_t N, int64_t K,
                   const int8_t *A, int64_t lda, const int8_t *W, int64_t ldw, int64_t stride_w,
                   void *C, int64_t ldc, const float *scale_a, const float *scale_w,
                   const float *bias, const int32_t *offsets, void *stream);

/*
 * The order of pairs by expert: a stable sort of `pairs` ids (id_type
 * MPGEMM_ID_*), equal experts in ascending pair order.
 *     order[p]     the pair at position p; -1 from offsets[experts] on
 *     position[i]  the position of pair i; -1 for a pair without an expert
 *     offsets[e]   the first position of expert e (experts + 1 values)
 * 1 <= experts <= MPGEMM_MAX_GROUPS, pairs <= 2^30.
 *
 * workspace: mpgemm_route_workspace(pairs, experts) bytes, 4-byte aligned
 * (NULL where that is 0; MPGEMM_ENULL or MPGEMM_EWORKSPACE otherwise).  Calls
 * that share one must not overlap in time.  mpgemm_route_workspace makes no
 * HIP call; it returns a negative code for sizes that mpgemm_route refuses.
 */
int64_t mpgemm_route_workspace(int64_t pairs, int64_t experts);

int mpgemm_route(int id_type, int64_t pairs, int64_t experts, const void *ids,
                 int32_t *order, int32_t *position, int32_t *offsets,
                 void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Rows into expert order:  Y[p] = X[order[p] / top_k],  p < R.
 * X: T x H, Y: R x H, both of `type`; rows whose order is outside 0 ..
 * T*top_k-1 keep what they hold.  workspace: see mpgemm_rows_workspace.  The
 * gradient by X is mpgemm_combine_rows of Y's gradient with weights NULL.
 */
int mpgemm_gather_rows(int type, int64_t T, int64_t H, const void *X, int64_t ldx,
                       const int32_t *order, int64_t R, int64_t top_k,
                       void *Y, int64_t ldy, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Workspace with which mpgemm_quantize_rows and mpgemm_gather_rows read each
 * token's row once when the rows in expert order are many: bytes, 4-byte
 * aligned, 0 where they do without.  A smaller one, or NULL, is no error: the
 * rows are then made one by one.  The results are the same.  Calls that share a workspace must
 * not overlap in time.  `type` is X's; no HIP call is made; a negative code
 * for arguments that those calls refuse.
 */
int64_t mpgemm_rows_workspace(int type, int64_t T, int64_t H, int64_t R, int64_t top_k);

/*
 * Experts' rows back to tokens:
 *     O[t] = sum_s weights[t][s] * Y[position[t][s]]
 * in FP32, slots ascending, rounded once to o_type.  Y: R x H of y_type, O:
 * T x H, position and weights (FP32; NULL: all 1) T x top_k, contiguous.  A
 * pair without a position adds nothing; a token without any has a row of
 * zeros.  top_k at most 2^30.
 */
int mpgemm_combine_rows(int y_type, int o_type, int64_t T, int64_t top_k, int64_t H, int64_t R,
                        const void *Y, int64_t ldy, const int32_t *position, const float *weights,
                        void *O, int64_t ldo, void *stream);

/*
 * The gradients of mpgemm_combine_rows from dO (T x H of d_type):
 *     dY[position[t][s]] = weights[t][s] * dO[t]           (dy_type)
 *     dweights[t][s]     = sum_h dO[t][h] * Y[position[t][s]][h]   (FP32)
 * Rows of dY that no pair has keep what they hold; dweights of a pair without
 * a position is 0.  dweights NULL: not computed, and Y is not read (it may be
 * NULL).  Positions must differ from pair to pair, as mpgemm_route makes them.
 */
int mpgemm_combine_rows_backward(int d_type, int y_type, int dy_type,
                                 int64_t T, int64_t top_k, int64_t H, int64_t R,
                                 const void *dO, int64_t ldo, const void *Y, int64_t ldy,
                                 const int32_t *position, const float *weights,
                                 void *dY, int64_t lddy, float *dweights, void *stream);

/*
 * The experts' 16-bit products: for every group g and its rows i,
 *     C[i][j] <- alpha * sum_k A[i][k] * B_g[k][j] + beta * C[i][j]
 * with the arithmetic, types and meaning of alpha and beta of mpgemm_gemm_ex.
 * A: R x K row-major, C: R x N FP32 row-major, B_g at B + g*stride_b, K x N
 * in storage order layout_b.  The gradient by A is this call on C's gradient
 * with B in the other storage order (N and K exchanged).
 * 128 stored rows of A, of one group's B and of C within 2 GiB (else
 * MPGEMM_ELD).  R, N and K below 2^31.
 */
int mpgemm_grouped(int in_type, int layout_b, int64_t groups, int64_t R, int64_t N, int64_t K,
                   const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb, int64_t stride_b,
                   float *C, int64_t ldc, float alpha, float beta,
                   const int32_t *offsets, void *stream);

/*
 * The same products' gradient by the weights: for every group g,
 *     C_g[i][j] <- alpha * sum_r A[r][i] * B[r][j] + beta * C_g[i][j]
 * over the group's rows r.  A: R x M and B: R x N row-major 16-bit, C_g at
 * C + g*stride_c, M x N FP32 row-major (stride_c >= the elements one spans).
 * A group without rows has C_g <- beta * C_g.  128 rows of A, B or C within
 * 2 GiB (else MPGEMM_ELD).
 */
int mpgemm_grouped_wgrad(int in_type, int64_t groups, int64_t R, int64_t M, int64_t N,
                         const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                         float *C, int64_t ldc, int64_t stride_c, float alpha, float beta,
                         const int32_t *offsets, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MPGEMM_OPS_H */
