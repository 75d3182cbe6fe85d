/*
 * mpgemm_router.h -- C ABI of the router in front of the experts, for gfx950
 * (AMD Instinct MI355X), in libmpgemm_router.so.
 *
 *   mpgemm_select_experts   the top_k experts of each token and their weights
 *   mpgemm_balance_loss     pairs and probabilities per expert, and the loss
 *                           that keeps them even
 *   mpgemm_router_backward  the gradient of both by the logits
 *
 * The rules of mpgemm_ops.h hold here too: device pointers the caller owns,
 * sizes and leading dimensions in elements, work enqueued on `stream`, nothing
 * allocated, kept or synchronized, 0 or a negative MPGEMM_E* code (argument
 * errors before any HIP call); every call may be recorded into a HIP graph;
 * results are the same from run to run; outputs must not overlap inputs or
 * each other; any element alignment.
 *
 * Logits: T x E of l_type (MPGEMM_T_*), ldl >= E; 1 <= E <= MPGEMM_MAX_GROUPS,
 * T below 2^31.  A token's probabilities are the softmax of its row in FP32:
 *     p[t][e] = exp(logits[t][e] - m) / sum_e exp(logits[t][e] - m),   m = max
 * A logit of -inf is an expert that the token may not have: its probability is
 * 0.  A row that is -inf throughout (a padding token) has probabilities 0 and
 * no expert.  A row that holds a NaN or +inf has NaN probabilities.
 *
 * Pairs: T x top_k, contiguous, as mpgemm_route takes them; an id outside 0 ..
 * E-1 is a pair without an expert.
 */
#ifndef MPGEMM_ROUTER_H
#define MPGEMM_ROUTER_H

#include <stdint.h>

#include "mpgemm_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest top_k of mpgemm_select_experts and mpgemm_router_backward. */
#define MPGEMM_MAX_SELECT 64

/*
 * Each token's top_k experts, by descending logit, equal ones by ascending
 * expert (a NaN stands before every number):
 *     ids[t][s]      the expert, or -1 where no expert is left but those at -inf
 *     weights[t][s]  normalize 0: p[t][ids[t][s]]
 *                    normalize 1: the same over their sum
 *                    (0 for a pair without an expert)
 * 1 <= top_k <= min(E, MPGEMM_MAX_SELECT).
 */
int mpgemm_select_experts(int l_type, int64_t T, int64_t E, int64_t top_k, int normalize,
                          const void *logits, int64_t ldl, int32_t *ids, float *weights, void *stream);

/*
 * How evenly the experts are used:
 *     counts[e]  the pairs of expert e, e < E
 *     counts[E]  the tokens that have probabilities (rows not -inf throughout)
 *     probs[e]   sum_t p[t][e]   (FP32; NULL: not written)
 *     loss       coefficient * E * sum_e counts[e] * probs[e] / (pairs * counts[E])
 * with pairs the sum of counts[e]; 0 where there are no pairs or no tokens.
 * Experts used evenly with even probabilities have loss = coefficient.  Sums
 * over tokens are FP32, in a fixed order.
 *
 * ids of id_type (MPGEMM_ID_*), T x top_k.  0 <= top_k, T*top_k below 2^31.
 * workspace: mpgemm_balance_workspace(T, E, top_k) bytes, 4-byte aligned
 * (MPGEMM_ENULL or MPGEMM_EWORKSPACE otherwise).  Calls that share one must not
 * overlap in time.  mpgemm_balance_workspace makes no HIP call; it returns a
 * negative code for sizes that mpgemm_balance_loss refuses.
 */
int64_t mpgemm_balance_workspace(int64_t T, int64_t E, int64_t top_k);

int mpgemm_balance_loss(int l_type, int id_type, int64_t T, int64_t E, int64_t top_k,
                        const void *logits, int64_t ldl, const void *ids, float coefficient,
                        float *loss, int32_t *counts, float *probs,
                        void *workspace, int64_t workspace_bytes, void *stream);

/*
 * The gradient by the logits of weights and loss, dlogits (T x E of d_type,
 * written whole, rounded once):
 *     u[t][e]  = sum over s with ids[t][s] == e of dweights[t][s]   (normalize 0)
 *              + dloss * coefficient * E * counts[e] / (pairs * counts[E])
 *     dlogits[t][e] = p[t][e] * (u[t][e] - sum_e p[t][e] * u[t][e])
 * and with normalize 1, w the weights of the pairs ids[t] in the softmax over
 * them alone, for each s
 *     dlogits[t][ids[t][s]] += w[t][s] * (dweights[t][s] - sum_s w[t][s] * dweights[t][s])
 * dweights NULL: the loss alone (ids is not read and may be NULL).  counts NULL:
 * the weights alone; otherwise as mpgemm_balance_loss wrote them, or their sums
 * over several devices.  dloss: one float in device memory, or NULL for 1.
 * ids may differ from those that mpgemm_select_experts chose.  A pair without an
 * expert, or whose expert's logit is -inf, has no part: its dweights may be
 * anything, infinities and NaN included.
 * top_k <= MPGEMM_MAX_SELECT.
 */
int mpgemm_router_backward(int l_type, int d_type, int id_type, int64_t T, int64_t E, int64_t top_k,
                           int normalize, const void *logits, int64_t ldl, const void *ids,
                           const float *dweights, const int32_t *counts, float coefficient,
                           const float *dloss, void *dlogits, int64_t ldd, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MPGEMM_ROUTER_H */
