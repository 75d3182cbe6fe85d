/*
 * mpgemm_ops_query.h -- which kernel a product of mpgemm_ops.h takes, for
 * tests and measurements (in libmpgemm_ops.so, beside the products).
 *
 * The choice depends on sizes and leading dimensions alone.  No HIP call is
 * made and no pointer but `out` is taken.  Return codes are those of the
 * product for the same arguments; a product without rows or columns launches
 * nothing and reports zeros.
 */
#ifndef MPGEMM_OPS_QUERY_H
#define MPGEMM_OPS_QUERY_H

#include <stdint.h>

#include "mpgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mpgemm_ops_kernel {
    int32_t narrow;      /* 1: 16 x 16 values a workgroup, whose waves split K and read
                          * their operands from memory; 0: tiles through LDS        */
    int32_t bm, bn;      /* values of C a workgroup makes                            */
    int32_t bk, stages;  /* values of K per tile in LDS, and tiles there (narrow: 0) */
    int32_t waves;       /* waves a workgroup                                        */
    int64_t workgroups;  /* launched: enough for any split of the rows into groups   */
} mpgemm_ops_kernel;

/* mpgemm_i8_gemm; groups 0: the call without offsets. */
int mpgemm_i8_query(int64_t groups, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldw,
                    mpgemm_ops_kernel *out);

/* mpgemm_grouped (the same for both input types). */
int mpgemm_grouped_query(int layout_b, int64_t groups, int64_t R, int64_t N, int64_t K,
                         int64_t lda, int64_t ldb, int64_t ldc, mpgemm_ops_kernel *out);

/* mpgemm_grouped_wgrad (the same for both input types). */
int mpgemm_grouped_wgrad_query(int64_t groups, int64_t R, int64_t M, int64_t N,
                               int64_t lda, int64_t ldb, int64_t ldc, mpgemm_ops_kernel *out);

#ifdef __cplusplus
}
#endif

#endif /* MPGEMM_OPS_QUERY_H */
