"""ctypes binding for libmpgemm_w4.so (include/mpgemm_w4.h): weights in 4-bit
codes with a scale per group of a row's values, and products with them.
Argument marshalling only, as in ``_binding``: every step runs in the HIP
library, there is no fallback."""
from __future__ import annotations

import ctypes
import os

from . import _ops
from ._binding import MPGEMM_OK, MpgemmError
from ._ops import MPGEMM_T_BF16, MPGEMM_T_F16, MpgemmOpsKernel, _call, _flat, _on, _rows, _type

W4_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmpgemm_w4.so")

_lib = None


def load_w4():
    """Load the in-tree libmpgemm_w4.so.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(W4_PATH):
        raise RuntimeError(f"{W4_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
                           "(no fallback path exists)")
    lib = ctypes.CDLL(W4_PATH)
    i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    for name, args in (
            ("mpgemm_w4_quantize", [i32, i32, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]),
            ("mpgemm_w4_dequantize", [i32, i32, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]),
            ("mpgemm_w4_gemm", [i32, i32, i64, i64, i64, i64, i64, vp, i64, vp, i64, i64, vp, i64, i64, vp, i64, vp, vp,
                                vp]),
            ("mpgemm_w4_query", [i64, i64, i64, i64, i64, i64, i64, i64, ctypes.POINTER(MpgemmOpsKernel)])):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = i32
    _lib = lib
    return lib


# ---- raw entry points (same names and argument order as the C ABI) ----------

def mpgemm_w4_quantize(w_type, s_type, N, K, group, W, ldw, Q, ldq, scale, lds, stream=0) -> int:
    return load_w4().mpgemm_w4_quantize(w_type, s_type, N, K, group, W, ldw, Q, ldq, scale, lds, stream)


def mpgemm_w4_dequantize(w_type, s_type, N, K, group, Q, ldq, scale, lds, W, ldw, stream=0) -> int:
    return load_w4().mpgemm_w4_dequantize(w_type, s_type, N, K, group, Q, ldq, scale, lds, W, ldw, stream)


def mpgemm_w4_gemm(in_type, out_type, groups, M, N, K, group, A, lda, Q, ldq, stride_q, scale, lds, stride_s, C, ldc,
                   bias=0, offsets=0, stream=0) -> int:
    return load_w4().mpgemm_w4_gemm(in_type, out_type, groups, M, N, K, group, A, lda, Q, ldq, stride_q, scale, lds,
                                    stride_s, C, ldc, bias, offsets, stream)


def mpgemm_w4_query(groups, M, N, K, group, lda, ldq, lds) -> dict:
    """The kernel that mpgemm_w4_gemm takes (groups 0: without offsets)."""
    out = MpgemmOpsKernel()
    rc = load_w4().mpgemm_w4_query(groups, M, N, K, group, lda, ldq, lds, ctypes.byref(out))
    if rc != MPGEMM_OK:
        raise MpgemmError(rc, "mpgemm_w4_query")
    return {field: getattr(out, field) for field, _ in out._fields_}


# ---- torch tensors ----------------------------------------------------------

_SCALES = (MPGEMM_T_F16, MPGEMM_T_BF16)


def _packed(Q, scale, N, K, group, types):
    """(pointer and leading dimension of Q, the same of scale, its type) of one
    matrix of N x K codes."""
    st = _type(scale, "scale", types)
    Nq, B, ldq = _rows(Q, "Q", _ops.torch.uint8)
    Ns, G, lds = _rows(scale, "scale", scale.dtype)
    if Nq != N or Ns != N or B != (K + 1) >> 1 or G != -(-K // group):
        raise ValueError(f"shape mismatch: Q {tuple(Q.shape)} and scale {tuple(scale.shape)} for {N} x {K} values in "
                         f"groups of {group}")
    return Q.data_ptr(), ldq, scale.data_ptr(), lds, st


def _group(group):
    group = int(group)
    if group < 1:
        raise ValueError("group must be a power of two, 32 or more")
    return group


def quantize_w4(W, Q, scale, group: int = 128, stream=None):
    """Rows of W to 4-bit codes, a scale for every ``group`` values of a row:
    scale = max|group| / 7 in the scale's type, and the codes of -8 .. 7 nearest
    to value / scale (ties to even).  Returns (Q, scale).

    W (N x K): float16, bfloat16 or float32, row-major.  Q (N x ceil(K / 2)):
    uint8, row-major; value k of a row is code + 8 in the low (even k) or high
    nibble of byte k // 2.  scale (N x ceil(K / group)): float16 or bfloat16,
    row-major.  group: a power of two, 32 or more.  A group with an infinity or
    a NaN has a NaN scale and codes 0."""
    if _ops.torch is None:
        _ops._with_torch()
    group = _group(group)
    wt = _type(W, "W")
    N, K, ldw = _rows(W, "W", W.dtype)
    qp, ldq, sp, lds, st = _packed(Q, scale, N, K, group, _SCALES)
    _call(load_w4().mpgemm_w4_quantize, _on(stream, W, Q, scale), wt, st, N, K, group, W.data_ptr(), ldw, qp, ldq, sp,
          lds)
    return Q, scale


def dequantize_w4(Q, scale, W, group: int = 128, stream=None):
    """W = code * scale: what :func:`quantize_w4` wrote, back as values, rounded
    once to W's type (float16, bfloat16 or float32).  Returns W."""
    if _ops.torch is None:
        _ops._with_torch()
    group = _group(group)
    wt = _type(W, "W")
    N, K, ldw = _rows(W, "W", W.dtype)
    qp, ldq, sp, lds, st = _packed(Q, scale, N, K, group, _SCALES)
    _call(load_w4().mpgemm_w4_dequantize, _on(stream, W, Q, scale), wt, st, N, K, group, qp, ldq, sp, lds,
          W.data_ptr(), ldw)
    return W


def _stacked(t, name, dtype, shape):
    """(leading dimension, stride of a matrix) of a 3-D GPU tensor of row-major
    matrices."""
    if not isinstance(t, _ops.torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {str(dtype).replace('torch.', '')} tensor")
    if tuple(t.shape) != shape:
        raise ValueError(f"shape mismatch: {name} {tuple(t.shape)}, expected {shape}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    sg, ld, step = t.stride()
    groups, rows, cols = shape
    ld = ld if rows > 1 else max(cols, 1)
    if (cols > 1 and step != 1) or ld < max(cols, 1):
        raise ValueError(f"{name}: its matrices must be row-major, their rows apart")
    return ld, (sg if groups > 1 else 0)


def gemm_w4(A, Q, scale, C, group: int = 128, bias=None, offsets=None, stream=None):
    """C <- A @ W.T (+ bias), W the values of 4-bit codes and scales; sums in
    FP32, no weight rounded.  Returns C.

    A (M x K): float16 or bfloat16, row-major.  Q (N x ceil(K / 2)): uint8 and
    scale (N x ceil(K / group)): of A's type, as :func:`quantize_w4` makes them.
    C (M x N): float16, bfloat16 or float32, row-major.  bias: float32, N values.
    With ``offsets`` (int32, groups + 1 values from :func:`route`) Q and scale
    have a matrix per group in front (bias: groups x N): rows offsets[g] ..
    offsets[g+1]-1 of A and C use group g's, other rows of C keep what they
    hold.  The gradient by A goes through :func:`dequantize_w4` to A's type (one
    rounding a weight) and ``gemm`` or ``gemm_grouped`` with the values."""
    if _ops.torch is None:
        _ops._with_torch()
    group = _group(group)
    it, ot = _type(A, "A", _SCALES), _type(C, "C")
    M, K, lda = _rows(A, "A", A.dtype)
    M2, N, ldc = _rows(C, "C", C.dtype)
    if M2 != M:
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, C {tuple(C.shape)}")
    if offsets is None:
        G, sq, ss, wide, op = 1, 0, 0, (N,), 0
        qp, ldq, sp, lds, _ = _packed(Q, scale, N, K, group, (it,))
    else:
        _type(scale, "scale", (it,))
        if not isinstance(Q, _ops.torch.Tensor) or Q.dim() != 3 or Q.shape[0] < 1:
            raise ValueError("Q must be groups x N x ceil(K / 2), at least one group")
        G = Q.shape[0]
        ldq, sq = _stacked(Q, "Q", _ops.torch.uint8, (G, N, (K + 1) // 2))
        lds, ss = _stacked(scale, "scale", A.dtype, (G, N, -(-K // group)))
        qp, sp, wide = Q.data_ptr(), scale.data_ptr(), (G, N)
        op = _flat(offsets, "offsets", _ops.torch.int32, (G + 1,))
    bp = 0 if bias is None else _flat(bias, "bias", _ops.torch.float32, wide)
    _call(load_w4().mpgemm_w4_gemm, _on(stream, C, A, Q, scale, bias, offsets), it, ot, G, M, N, K, group,
          A.data_ptr(), lda, qp, ldq, sq, sp, lds, ss, C.data_ptr(), ldc, bp, op)
    return C
