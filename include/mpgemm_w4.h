/*
 * mpgemm_w4.h -- C ABI of 4-bit weights with a scale per group of a row's
 * values, for gfx950 (AMD Instinct MI355X), in libmpgemm_w4.so.
 *
 *   mpgemm_w4_quantize     rows of weights to codes and scales
 *   mpgemm_w4_dequantize   and back to values
 *   mpgemm_w4_gemm         product of 16-bit tokens with such weights, one
 *                          matrix or one per expert
 *   mpgemm_w4_query        the kernel that such a product takes (host only)
 *
 * The rules of mpgemm_ops.h hold here too: device pointers the caller owns,
 * sizes and leading dimensions in elements, work enqueued on `stream`, nothing
 * allocated, kept or synchronized, 0 or a negative MPGEMM_E* code (argument
 * errors before any HIP call); every call may be recorded into a HIP graph;
 * results are the same from run to run; outputs must not overlap inputs or
 * each other; any size >= 0 within the limits and any element alignment.
 *
 * Format.  N rows (channels) of K values.  A row's values k*group ..
 * (k+1)*group - 1 share scale k (the last group may be short); `group` is a
 * power of two from 32 to 2^28.  A code is a whole number c of -8 .. 7 and stands
 * in four bits as c + 8; value k of a row is the low nibble of byte k/2 where k
 * is even, the high one where it is odd.  The value is c * scale.
 *     Q:     N x ceil(K/2) bytes,       ldq >= max(1, ceil(K/2))
 *     scale: N x ceil(K/group) of s_type (MPGEMM_T_F16 or MPGEMM_T_BF16),
 *            lds >= max(1, ceil(K/group))
 * The spare nibble of a row of odd K is written as 8 and not looked at.
 * K at most 2^28, N below 2^31.
 */
#ifndef MPGEMM_W4_H
#define MPGEMM_W4_H

#include <stdint.h>

#include "mpgemm_ops.h"
#include "mpgemm_ops_query.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Weights to codes.  For each group, with m its largest magnitude:
 *     scale = m / 7, rounded to FP32 and then to s_type
 *     code  = the whole number of -8 .. 7 nearest to value / scale (the exact
 *             quotient; the even one in the middle)
 * A group whose scale is 0 has codes 0.  A group that holds an infinity or a
 * NaN, or whose scale s_type does not hold, has a NaN scale and codes 0: what
 * is made of it is NaN.
 * W: N x K of w_type (MPGEMM_T_*), ldw >= max(1,K).
 */
int mpgemm_w4_quantize(int w_type, int s_type, int64_t N, int64_t K, int64_t group,
                       const void *W, int64_t ldw, uint8_t *Q, int64_t ldq,
                       void *scale, int64_t lds, void *stream);

/* Back to values:  W[j][k] = code * scale, rounded once to w_type. */
int mpgemm_w4_dequantize(int w_type, int s_type, int64_t N, int64_t K, int64_t group,
                         const uint8_t *Q, int64_t ldq, const void *scale, int64_t lds,
                         void *W, int64_t ldw, void *stream);

/*
 * Product of tokens with 4-bit weights:
 *     C[i][j] = sum_g scale[j][g] * (sum_{k in g} A[i][k] * code[j][k]) (+ bias[j])
 * The codes are multiplied exactly; the sum of up to 128 of a group's products
 * (128: of larger groups too) is FP32 and joins the FP32 sum of a row by one
 * fused multiply-add with its scale; the bias is added in FP32; out_type rounds
 * once.  No weight is rounded.  Those sums come before the scale: BF16 tokens of
 * magnitude 2^122 (5.3e36) or more may overflow there although the scaled result
 * would not; smaller ones, and FP16 ones, cannot.
 *
 * A: M x K of in_type (MPGEMM_IN_F16 or MPGEMM_IN_BF16), lda >= max(1,K).
 * Q, scale: as above, scale of the same type as A.  C: M x N of out_type
 * (MPGEMM_T_*), ldc >= max(1,N).  bias: N floats or NULL.
 *
 * offsets NULL: one product, groups must be 1.  Otherwise rows offsets[g] ..
 * offsets[g+1]-1 of A and C use the codes at Q + g*stride_q, the scales at
 * scale + g*stride_s and row g of bias (groups x N, contiguous); rows of C that
 * no group has keep what they hold.  See mpgemm_ops.h for offsets and groups.
 *
 * The gradient by the tokens, dA = dC * W, has no call of its own: it is
 * mpgemm_w4_dequantize to in_type (each weight code * scale rounded once, half a
 * step of that type, which the product above does not do) and the 16-bit product
 * with the values (mpgemm_gemm_ex; per expert mpgemm_grouped).
 *
 * M below 2^31; 64 rows of A, and 32 rows of Q and of scale, within 2 GiB
 * (else MPGEMM_ELD); at most 2^22 tiles (else MPGEMM_EDIM).
 */
int mpgemm_w4_gemm(int in_type, int out_type, int64_t groups, int64_t M, int64_t N, int64_t K, int64_t group,
                   const uint16_t *A, int64_t lda, const uint8_t *Q, int64_t ldq, int64_t stride_q,
                   const void *scale, int64_t lds, int64_t stride_s, void *C, int64_t ldc,
                   const float *bias, const int32_t *offsets, void *stream);

/* The kernel that mpgemm_w4_gemm takes, from sizes and leading dimensions
 * alone; groups 0: the call without offsets.  The same for all types. */
int mpgemm_w4_query(int64_t groups, int64_t M, int64_t N, int64_t K, int64_t group,
                    int64_t lda, int64_t ldq, int64_t lds, mpgemm_ops_kernel *out);

#ifdef __cplusplus
}
#endif

#endif /* MPGEMM_W4_H */
