"""ctypes binding for libmpgemm_router.so (include/mpgemm_router.h): the
router in front of the experts.  Argument marshalling only, as in
``_binding``: every step runs in the HIP library, there is no fallback."""
from __future__ import annotations

import ctypes
import os

from . import _ops
from ._binding import MpgemmError
from ._ops import MPGEMM_ID_I32, MPGEMM_ID_I64, _call, _check_workspace, _flat, _on, _type, _workspace

ROUTER_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmpgemm_router.so")
#: largest top_k of select_experts and router_backward
MPGEMM_MAX_SELECT = 64

_lib = None


def load_router():
    """Load the in-tree libmpgemm_router.so.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(ROUTER_PATH):
        raise RuntimeError(f"{ROUTER_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
                           "(no fallback path exists)")
    lib = ctypes.CDLL(ROUTER_PATH)
    i64, f32, vp, i32 = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int
    for name, args, res in (
            ("mpgemm_select_experts", [i32, i64, i64, i64, i32, vp, i64, vp, vp, vp], i32),
            ("mpgemm_balance_workspace", [i64, i64, i64], i64),
            ("mpgemm_balance_loss", [i32, i32, i64, i64, i64, vp, i64, vp, f32, vp, vp, vp, vp, i64, vp], i32),
            ("mpgemm_router_backward",
             [i32, i32, i32, i64, i64, i64, i32, vp, i64, vp, vp, vp, f32, vp, vp, i64, vp], i32)):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


# ---- raw entry points (same names and argument order as the C ABI) ----------

def mpgemm_select_experts(l_type, T, E, top_k, normalize, logits, ldl, ids, weights, stream=0) -> int:
    return load_router().mpgemm_select_experts(l_type, T, E, top_k, normalize, logits, ldl, ids, weights, stream)


def mpgemm_balance_workspace(T, E, top_k) -> int:
    """Bytes of workspace that mpgemm_balance_loss needs, or a negative code."""
    return load_router().mpgemm_balance_workspace(T, E, top_k)


def mpgemm_balance_loss(l_type, id_type, T, E, top_k, logits, ldl, ids, coefficient, loss, counts, probs, workspace,
                        workspace_bytes, stream=0) -> int:
    return load_router().mpgemm_balance_loss(l_type, id_type, T, E, top_k, logits, ldl, ids, coefficient, loss, counts,
                                             probs, workspace, workspace_bytes, stream)


def mpgemm_router_backward(l_type, d_type, id_type, T, E, top_k, normalize, logits, ldl, ids, dweights, counts,
                           coefficient, dloss, dlogits, ldd, stream=0) -> int:
    return load_router().mpgemm_router_backward(l_type, d_type, id_type, T, E, top_k, normalize, logits, ldl, ids,
                                                dweights, counts, coefficient, dloss, dlogits, ldd, stream)


# ---- torch tensors ----------------------------------------------------------

def _logits(t, name):
    """(type, tokens, experts, leading dimension) of a row-major 2-D tensor."""
    ty = _type(t, name)
    T, E, ld = _ops._rows(t, name, t.dtype)
    return ty, T, E, ld


def _ids(ids, T):
    """(type, pointer, top_k) of the pairs' experts."""
    if not isinstance(ids, _ops.torch.Tensor) or ids.dtype not in (_ops.torch.int32, _ops.torch.int64):
        raise TypeError("ids must be an int32 or int64 tensor")
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids must be {T} x top_k, got {tuple(ids.shape)}")
    if not ids.is_cuda or not ids.is_contiguous():
        raise ValueError("ids must be contiguous, on the GPU")
    return MPGEMM_ID_I64 if ids.dtype == _ops.torch.int64 else MPGEMM_ID_I32, ids.data_ptr(), ids.shape[1]


def select_experts(logits, ids, weights, normalize: bool = True, stream=None):
    """Each token's experts by the softmax of its logits: ids[t, s] is the
    expert with the (s + 1)-th largest logit (equal ones in ascending order),
    weights[t, s] its probability, or with ``normalize`` its share of the chosen
    ones' sum.  Returns (ids, weights).

    logits (T x experts): float16, bfloat16 or float32, row-major.  ids (T x
    top_k): int32, and weights: float32, contiguous; top_k at most 64.  An expert
    whose logit is -inf is never chosen: where no other is left the id is -1 and
    the weight 0, a pair without an expert for :func:`route`."""
    if _ops.torch is None:
        _ops._with_torch()
    lt, T, E, ldl = _logits(logits, "logits")
    if not isinstance(ids, _ops.torch.Tensor) or ids.dim() != 2:
        raise ValueError(f"ids must be {T} x top_k")
    shape = (T, ids.shape[1])
    ip = _flat(ids, "ids", _ops.torch.int32, shape)
    wp = _flat(weights, "weights", _ops.torch.float32, shape)
    _call(load_router().mpgemm_select_experts, _on(stream, logits, ids, weights), lt, T, E, shape[1],
          1 if normalize else 0, logits.data_ptr(), ldl, ip, wp)
    return ids, weights


def balance_loss(logits, ids, loss, counts, probs=None, coefficient: float = 1.0, workspace=None, stream=None):
    """How evenly the experts are used, and the loss that evens it:
    coefficient * experts * sum_e counts[e] * probs[e] / (pairs * tokens).
    Returns (loss, counts).

    logits (T x experts): float16, bfloat16 or float32, row-major.  ids (T x
    top_k): int32 or int64, contiguous; pairs outside 0 .. experts-1 count for
    none.  loss: float32, 1 value.  counts: int32, experts + 1 values: the pairs
    of each expert, then the tokens whose logits are not -inf throughout.  probs:
    float32, experts values or None: the sum over the tokens of each expert's
    probability.  ``workspace``: a contiguous int32 tensor of
    mpgemm_balance_workspace bytes; allocated when None.  The gradient is
    :func:`router_backward` with ``counts``."""
    if _ops.torch is None:
        _ops._with_torch()
    _check_workspace(workspace)
    lt, T, E, ldl = _logits(logits, "logits")
    it, ip, k = _ids(ids, T)
    lp = _flat(loss, "loss", _ops.torch.float32, (1,))
    cp = _flat(counts, "counts", _ops.torch.int32, (E + 1,))
    pp = 0 if probs is None else _flat(probs, "probs", _ops.torch.float32, (E,))
    lib = load_router()
    need = lib.mpgemm_balance_workspace(T, E, k)
    if need < 0:
        raise MpgemmError(need, "mpgemm_balance_loss")
    on = _on(stream, logits, ids, loss, counts, probs, workspace)
    wp, wb, _ws = _workspace(on, stream, workspace, need)
    _call(lib.mpgemm_balance_loss, on, lt, it, T, E, k, logits.data_ptr(), ldl, ip, float(coefficient), lp, cp, pp, wp,
          wb)
    return loss, counts


def router_backward(logits, ids, dlogits, dweights=None, normalize: bool = True, counts=None, dloss=None,
                    coefficient: float = 1.0, stream=None):
    """The gradient by the logits of :func:`select_experts`' weights
    (``dweights``, with the same ``normalize``) and of :func:`balance_loss`
    (``counts`` as it wrote them, the same ``coefficient``, ``dloss`` the loss's
    own gradient), of either or of both.  Writes dlogits and returns it.

    logits and dlogits (T x experts): float16, bfloat16 or float32 each,
    row-major.  ids (T x top_k): int32 or int64, contiguous; None without
    dweights.  dweights: float32, T x top_k; what it holds at a pair without an
    expert, or of one whose logit is -inf, is not used.  counts: int32, experts +
    1 values, summed over devices where tokens are spread.  dloss: float32, 1 value, or
    None for 1."""
    if _ops.torch is None:
        _ops._with_torch()
    lt, T, E, ldl = _logits(logits, "logits")
    dt, T2, E2, ldd = _logits(dlogits, "dlogits")
    if T2 != T or E2 != E:
        raise ValueError(f"shape mismatch: logits {tuple(logits.shape)}, dlogits {tuple(dlogits.shape)}")
    it, ip, k, wp = MPGEMM_ID_I32, 0, 0, 0
    if dweights is not None:
        if ids is None:
            raise ValueError("dweights needs ids")
        it, ip, k = _ids(ids, T)
        wp = _flat(dweights, "dweights", _ops.torch.float32, (T, k))
    cp = 0 if counts is None else _flat(counts, "counts", _ops.torch.int32, (E + 1,))
    lp = 0 if dloss is None else _flat(dloss, "dloss", _ops.torch.float32, (1,))
    _call(load_router().mpgemm_router_backward,
          _on(stream, dlogits, logits, None if dweights is None else ids, dweights, counts, dloss), lt, dt, it, T, E, k,
          1 if normalize else 0, logits.data_ptr(), ldl, ip, wp, cp, float(coefficient), lp, dlogits.data_ptr(), ldd)
    return dlogits
