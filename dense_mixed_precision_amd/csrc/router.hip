// router.hip -- host side of the router's operators (include/mpgemm_router.h):
// argument validation, launches.
#include "mpgemm_router.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#define mpg mpg_router
namespace mpg {
#include "elements.hpp"
#include "router_kernels.hpp"
}  // namespace mpg

#include "host_util.hpp"

namespace {

using mpg::BalanceArgs;
using mpg::RouterArgs;
using mpg::RouterBackArgs;

// Calls f with the lanes of a token and the values of each, the fewest that
// hold a row (and, where they matter, a lane per slot).
template <class F>
void by_width(int64_t E, int64_t slots, F f)
{
    using std::integral_constant;
    if (E <= 256 && slots <= 16) {
        if (E <= 16)
            f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
        else if (E <= 32)
            f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
        else if (E <= 64)
            f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
        else if (E <= 128)
            f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
        else
            f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
    } else if (E <= 256) {
        f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    } else if (E <= 512) {
        f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
    } else {
        f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
    }
}

// Calls f with a type as a constant.
template <class F>
void by_type(int type, F f)
{
    if (type == MPGEMM_T_F16)
        f(std::integral_constant<int, mpg::kTF16>{});
    else if (type == MPGEMM_T_BF16)
        f(std::integral_constant<int, mpg::kTBF16>{});
    else
        f(std::integral_constant<int, mpg::kTF32>{});
}

int check_logits(int l_type, int64_t T, int64_t E, int64_t ldl)
{
    if (!is_type(l_type))
        return MPGEMM_ETYPE;
    if (T < 0 || T > kMax32 || E < 1 || E > MPGEMM_MAX_GROUPS)
        return MPGEMM_EDIM;
    return ldl < E ? MPGEMM_ELD : MPGEMM_OK;
}

bool is_id(int t) { return t == MPGEMM_ID_I32 || t == MPGEMM_ID_I64; }
int64_t id_size(int t) { return t == MPGEMM_ID_I64 ? 8 : 4; }

// Blocks of the first launch of the loss and tokens of each: blocks for every
// compute unit twice, of 64 tokens at least.
struct BalancePlan {
    int64_t blocks, per_block;
};

BalancePlan plan_balance(int64_t T)
{
    int64_t blocks = cdiv(T, 64);
    blocks = blocks > 2 * kNumCu ? 2 * kNumCu : blocks < 1 ? 1 : blocks;
    const int64_t per = cdiv(cdiv(T, blocks), 16) * 16;
    return BalancePlan{T == 0 ? 1 : cdiv(T, per), per};
}

int64_t balance_sums(int64_t E) { return cdiv(E + 1, mpg::kBalanceExperts); }

}  // namespace

extern "C" {

int mpgemm_select_experts(int l_type, int64_t T, int64_t E, int64_t top_k, int normalize,
                          const void *logits, int64_t ldl, int32_t *ids, float *weights, void *stream)
{
    if (const int error = check_logits(l_type, T, E, ldl))
        return error;
    if (top_k < 1 || top_k > E || top_k > MPGEMM_MAX_SELECT)
        return MPGEMM_EDIM;
    if (T == 0)
        return MPGEMM_OK;
    if (logits == nullptr || ids == nullptr || weights == nullptr)
        return MPGEMM_ENULL;
    if (!aligned(logits, size_of(l_type)) || !aligned(ids, 4) || !aligned(weights, 4))
        return MPGEMM_EALIGN;
    const RouterArgs a{logits, ldl, (int32_t)T, (int32_t)E, (int32_t)top_k};
    forget_error();
    by_type(l_type, [&](auto lt) {
        by_width(E, top_k, [&](auto lpt, auto v) {
            hipLaunchKernelGGL((mpg::select_experts<lt.value, lpt.value, v.value>), row_grid(cdiv(T, 256 / lpt.value)),
                               dim3(256), 0, stream_of(stream), a, normalize != 0, ids, weights);
        });
    });
    return launched();
}

int64_t mpgemm_balance_workspace(int64_t T, int64_t E, int64_t top_k)
{
    if (T < 0 || T > kMax32 || E < 1 || E > MPGEMM_MAX_GROUPS || top_k < 0 || mul_sat(T, top_k) > kMax32)
        return MPGEMM_EDIM;
    return 4 * (plan_balance(T).blocks * (2 * E + 1) + 1 + 3 * balance_sums(E));
}

int mpgemm_balance_loss(int l_type, int id_type, int64_t T, int64_t E, int64_t top_k,
                        const void *logits, int64_t ldl, const void *ids, float coefficient,
                        float *loss, int32_t *counts, float *probs,
                        void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!is_id(id_type))
        return MPGEMM_ETYPE;
    if (const int error = check_logits(l_type, T, E, ldl))
        return error;
    const int64_t need = mpgemm_balance_workspace(T, E, top_k);
    if (need < 0)
        return MPGEMM_EDIM;
    if (loss == nullptr || counts == nullptr || workspace == nullptr || (T > 0 && logits == nullptr) ||
        (T > 0 && top_k > 0 && ids == nullptr))
        return MPGEMM_ENULL;
    if (!aligned(logits, size_of(l_type)) || !aligned(ids, id_size(id_type)) || !aligned(loss, 4) ||
        !aligned(counts, 4) || !aligned(probs, 4) || !aligned(workspace, 4))
        return MPGEMM_EALIGN;
    if (workspace_bytes < need)
        return MPGEMM_EWORKSPACE;
    const BalancePlan plan = plan_balance(T);
    const BalanceArgs a{RouterArgs{logits, ldl, (int32_t)T, (int32_t)E, (int32_t)top_k},
                        ids, coefficient, loss, probs, counts, static_cast<uint32_t *>(workspace),
                        (int32_t)plan.blocks, (int32_t)plan.per_block};
    forget_error();
    by_type(l_type, [&](auto lt) {
        by_width(E, 0, [&](auto lpt, auto v) {
            const size_t lds = 4 * (size_t)(E + 1 + 4 * lpt.value * v.value);
            if (id_type == MPGEMM_ID_I64)
                hipLaunchKernelGGL((mpg::balance_tokens<lt.value, lpt.value, v.value, 1>), dim3((unsigned)plan.blocks),
                                   dim3(256), lds, stream_of(stream), a);
            else
                hipLaunchKernelGGL((mpg::balance_tokens<lt.value, lpt.value, v.value, 0>), dim3((unsigned)plan.blocks),
                                   dim3(256), lds, stream_of(stream), a);
        });
    });
    if (const int error = launched())
        return error;
    hipLaunchKernelGGL(mpg::balance_sum, dim3((unsigned)balance_sums(E)), dim3(1024), 0, stream_of(stream), a);
    return launched();
}

int mpgemm_router_backward(int l_type, int d_type, int id_type, int64_t T, int64_t E, int64_t top_k,
                           int normalize, const void *logits, int64_t ldl, const void *ids,
                           const float *dweights, const int32_t *counts, float coefficient,
                           const float *dloss, void *dlogits, int64_t ldd, void *stream)
{
    if (!is_type(d_type) || !is_id(id_type))
        return MPGEMM_ETYPE;
    if (const int error = check_logits(l_type, T, E, ldl))
        return error;
    if (top_k < 0 || top_k > MPGEMM_MAX_SELECT)
        return MPGEMM_EDIM;
    if (ldd < E)
        return MPGEMM_ELD;
    if (T == 0)
        return MPGEMM_OK;
    if (logits == nullptr || dlogits == nullptr || (dweights != nullptr && top_k > 0 && ids == nullptr))
        return MPGEMM_ENULL;
    if (!aligned(logits, size_of(l_type)) || !aligned(dlogits, size_of(d_type)) || !aligned(ids, id_size(id_type)) ||
        !aligned(dweights, 4) || !aligned(counts, 4) || !aligned(dloss, 4))
        return MPGEMM_EALIGN;
    const RouterBackArgs a{RouterArgs{logits, ldl, (int32_t)T, (int32_t)E, (int32_t)top_k},
                           ids, dweights, counts, dloss, coefficient, normalize != 0, dlogits, ldd};
    forget_error();
    by_type(l_type, [&](auto lt) {
        by_type(d_type, [&](auto dt) {
            by_width(E, dweights ? top_k : 0, [&](auto lpt, auto v) {
                const int64_t blocks = cdiv(T, 256 / lpt.value);
                const dim3 grid((unsigned)(blocks < 8 * kNumCu ? blocks : 8 * kNumCu));
                if (id_type == MPGEMM_ID_I64)
                    hipLaunchKernelGGL((mpg::router_backward<lt.value, dt.value, lpt.value, v.value, 1>), grid,
                                       dim3(256), 0, stream_of(stream), a);
                else
                    hipLaunchKernelGGL((mpg::router_backward<lt.value, dt.value, lpt.value, v.value, 0>), grid,
                                       dim3(256), 0, stream_of(stream), a);
            });
        });
    });
    return launched();
}

}  // extern "C"
