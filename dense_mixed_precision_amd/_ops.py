"""ctypes binding for libmpgemm_ops.so (include/mpgemm_ops.h and
mpgemm_ops_query.h): products of 8-bit codes and products of tokens with
experts.  Argument marshalling only, as in ``_binding``: every step runs in
the HIP library, there is no fallback."""
from __future__ import annotations

import ctypes
import os

from ._binding import MPGEMM_COL_MAJOR, MPGEMM_OK, MPGEMM_ROW_MAJOR, MpgemmError, _check_tensor

OPS_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmpgemm_ops.so")

MPGEMM_T_F16 = 0
MPGEMM_T_BF16 = 1
MPGEMM_T_F32 = 2
MPGEMM_ID_I32 = 0
MPGEMM_ID_I64 = 1
#: groups (experts) of one grouped call
MPGEMM_MAX_GROUPS = 1024
#: largest K of mpgemm_i8_gemm
MPGEMM_I8_MAX_K = 131071



class MpgemmOpsKernel(ctypes.Structure):
    """mpgemm_ops_kernel of include/mpgemm_ops_query.h."""
    _fields_ = [*((n, ctypes.c_int32) for n in ("narrow", "bm", "bn", "bk", "stages", "waves")),
                ("workgroups", ctypes.c_int64)]


_lib = None
#: torch, imported by the first call that takes tensors (the raw entry points
#: need none); not by an import in each function, which a small launch notices
torch = None


def _with_torch():
    global torch, _TYPES
    import torch as module
    # torch last: another thread's first call takes its presence for all of this
    _TYPES = {module.float16: MPGEMM_T_F16, module.bfloat16: MPGEMM_T_BF16, module.float32: MPGEMM_T_F32}
    torch = module


def load_ops():
    """Load the in-tree libmpgemm_ops.so.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(OPS_PATH):
        raise RuntimeError(f"{OPS_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
                           "(no fallback path exists)")
    lib = ctypes.CDLL(OPS_PATH)
    i64, f32, vp, i32 = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int
    kernel = ctypes.POINTER(MpgemmOpsKernel)
    for name, args, res in (
            ("mpgemm_quantize_rows", [i32, i64, i64, vp, i64, vp, i64, i64, vp, i64, vp, vp, i64, vp], i32),
            ("mpgemm_rows_workspace", [i32, i64, i64, i64, i64], i64),
            ("mpgemm_i8_gemm", [i32, i64, i64, i64, i64, vp, i64, vp, i64, i64, vp, i64, vp, vp, vp, vp, vp], i32),
            ("mpgemm_route_workspace", [i64, i64], i64),
            ("mpgemm_route", [i32, i64, i64, vp, vp, vp, vp, vp, i64, vp], i32),
            ("mpgemm_gather_rows", [i32, i64, i64, vp, i64, vp, i64, i64, vp, i64, vp, i64, vp], i32),
            ("mpgemm_combine_rows", [i32, i32, i64, i64, i64, i64, vp, i64, vp, vp, vp, i64, vp], i32),
            ("mpgemm_combine_rows_backward",
             [i32, i32, i32, i64, i64, i64, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, vp], i32),
            ("mpgemm_grouped", [i32, i32, i64, i64, i64, i64, vp, i64, vp, i64, i64, vp, i64, f32, f32, vp, vp], i32),
            ("mpgemm_grouped_wgrad", [i32, i64, i64, i64, i64, vp, i64, vp, i64, vp, i64, i64, f32, f32, vp, vp], i32),
            ("mpgemm_i8_query", [i64, i64, i64, i64, i64, i64, kernel], i32),
            ("mpgemm_grouped_query", [i32, i64, i64, i64, i64, i64, i64, i64, kernel], i32),
            ("mpgemm_grouped_wgrad_query", [i64, i64, i64, i64, i64, i64, i64, kernel], i32)):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


# ---- raw entry points (same names and argument order as the C ABI) ----------

def mpgemm_quantize_rows(x_type, T, H, X, ldx, order, R, top_k, Q, ldq, scale, workspace=0, workspace_bytes=0,
                         stream=0) -> int:
    return load_ops().mpgemm_quantize_rows(x_type, T, H, X, ldx, order, R, top_k, Q, ldq, scale, workspace,
                                           workspace_bytes, stream)


def mpgemm_rows_workspace(type_, T, H, R, top_k) -> int:
    """Bytes of workspace that lets mpgemm_quantize_rows and mpgemm_gather_rows
    read each token once, 0 if none does, or a negative code."""
    return load_ops().mpgemm_rows_workspace(type_, T, H, R, top_k)


def mpgemm_i8_gemm(out_type, groups, M, N, K, A, lda, W, ldw, stride_w, C, ldc, scale_a, scale_w, bias=0,
                   offsets=0, stream=0) -> int:
    return load_ops().mpgemm_i8_gemm(out_type, groups, M, N, K, A, lda, W, ldw, stride_w, C, ldc, scale_a, scale_w,
                                     bias, offsets, stream)


def mpgemm_route_workspace(pairs, experts) -> int:
    """Bytes of workspace that mpgemm_route needs, or a negative code."""
    return load_ops().mpgemm_route_workspace(pairs, experts)


def mpgemm_route(id_type, pairs, experts, ids, order, position, offsets, workspace=0, workspace_bytes=0,
                 stream=0) -> int:
    return load_ops().mpgemm_route(id_type, pairs, experts, ids, order, position, offsets, workspace,
                                   workspace_bytes, stream)


def mpgemm_gather_rows(type_, T, H, X, ldx, order, R, top_k, Y, ldy, workspace=0, workspace_bytes=0,
                       stream=0) -> int:
    return load_ops().mpgemm_gather_rows(type_, T, H, X, ldx, order, R, top_k, Y, ldy, workspace, workspace_bytes,
                                         stream)


def mpgemm_combine_rows(y_type, o_type, T, top_k, H, R, Y, ldy, position, weights, O, ldo, stream=0) -> int:
    return load_ops().mpgemm_combine_rows(y_type, o_type, T, top_k, H, R, Y, ldy, position, weights, O, ldo, stream)


def mpgemm_combine_rows_backward(d_type, y_type, dy_type, T, top_k, H, R, dO, ldo, Y, ldy, position, weights, dY,
                                 lddy, dweights, stream=0) -> int:
    return load_ops().mpgemm_combine_rows_backward(d_type, y_type, dy_type, T, top_k, H, R, dO, ldo, Y, ldy,
                                                   position, weights, dY, lddy, dweights, stream)


def mpgemm_grouped(in_type, layout_b, groups, R, N, K, A, lda, B, ldb, stride_b, C, ldc, alpha, beta, offsets,
                   stream=0) -> int:
    return load_ops().mpgemm_grouped(in_type, layout_b, groups, R, N, K, A, lda, B, ldb, stride_b, C, ldc, alpha,
                                     beta, offsets, stream)


def mpgemm_grouped_wgrad(in_type, groups, R, M, N, A, lda, B, ldb, C, ldc, stride_c, alpha, beta, offsets,
                         stream=0) -> int:
    return load_ops().mpgemm_grouped_wgrad(in_type, groups, R, M, N, A, lda, B, ldb, C, ldc, stride_c, alpha, beta,
                                           offsets, stream)


def _query(name, *args) -> dict:
    out = MpgemmOpsKernel()
    rc = getattr(load_ops(), name)(*args, ctypes.byref(out))
    if rc != MPGEMM_OK:
        raise MpgemmError(rc, name)
    return {field: getattr(out, field) for field, _ in out._fields_}


def mpgemm_i8_query(groups, M, N, K, lda, ldw) -> dict:
    """The kernel that mpgemm_i8_gemm takes (groups 0: without offsets)."""
    return _query("mpgemm_i8_query", groups, M, N, K, lda, ldw)


def mpgemm_grouped_query(layout_b, groups, R, N, K, lda, ldb, ldc) -> dict:
    return _query("mpgemm_grouped_query", layout_b, groups, R, N, K, lda, ldb, ldc)


def mpgemm_grouped_wgrad_query(groups, R, M, N, lda, ldb, ldc) -> dict:
    return _query("mpgemm_grouped_wgrad_query", groups, R, M, N, lda, ldb, ldc)


# ---- torch tensors ----------------------------------------------------------

_TYPES: dict = {}


def _type(t, name, types=(MPGEMM_T_F16, MPGEMM_T_BF16, MPGEMM_T_F32)):
    """MPGEMM_T_* of a tensor's dtype, one of `types`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _TYPES.get(t.dtype)
    if code not in types:
        names = [str(d).replace("torch.", "") for d, c in _TYPES.items() if c in types]
        raise TypeError(f"{name} must be {' or '.join(names)}, got {t.dtype}")
    return code


def _rows(t, name, dtype):
    """(rows, columns, leading dimension) of a row-major 2-D GPU tensor."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.dim() == 2:
        # the ordinary case at once; the rest, and what is refused, below
        ld, step = t.stride()
        rows, cols = t.shape
        if step == 1 and rows > 1 and ld >= cols > 0:
            return rows, cols, ld
    ld = _check_tensor(t, name, dtype)[1]
    return t.shape[0], t.shape[1], ld


def _flat(t, name, dtype, shape):
    """Pointer of a contiguous GPU tensor of one dtype and shape (None: any)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {str(dtype).replace('torch.', '')} tensor")
    if (shape is not None and t.shape != shape) or not t.is_contiguous():
        want = "" if shape is None else f", of shape {tuple(shape)}, got {tuple(t.shape)}"
        raise ValueError(f"{name} must be contiguous{want}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    return t.data_ptr()


def _matrices(t, name, dtype):
    """(groups, rows, cols, layout, leading dimension, group stride) of a 3-D
    GPU tensor of matrices, each row- or column-major."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {str(dtype).replace('torch.', '')} tensor")
    if t.dim() != 3 or t.shape[0] < 1:
        raise ValueError(f"{name} must be groups x rows x columns, at least one group")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    groups, rows, cols = t.shape
    sg, sr, sc = t.stride()
    if cols <= 1 or sc == 1:
        layout, ld, least = MPGEMM_ROW_MAJOR, (sr if rows > 1 else max(cols, 1)), cols
    elif rows <= 1 or sr == 1:
        layout, ld, least = MPGEMM_COL_MAJOR, sc, rows
    else:
        raise ValueError(f"{name}: its matrices must have unit stride along one dimension")
    if ld < max(least, 1):
        raise ValueError(f"{name}: the rows or columns of its matrices overlap (stride {ld} < {least})")
    return groups, rows, cols, layout, ld, (sg if groups > 1 else 0)


def _check_workspace(t):
    if t is not None and (not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or not t.is_contiguous()):
        raise TypeError("workspace must be a contiguous int32 tensor on the GPU")


def _on(stream, *tensors):
    """(device index, stream handle) of a call: every tensor on one GPU, the
    launch on that GPU's current stream or the one given."""
    device = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"tensors are on {tensors[0].device} and {t.device}: one GPU is needed")
    if stream is None:
        # the handle alone: a Stream object costs as much as a small launch
        return device, torch._C._cuda_getCurrentRawStream(device)
    if hasattr(stream, "cuda_stream"):
        if stream.device.index != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {tensors[0].device}")
        return device, stream.cuda_stream
    return device, int(stream)


def _new(on, stream, *shapes):
    """Uninitialised int32 tensors that belong to the launch's stream: memory
    that another stream freed may still be in use there."""
    device = torch.device("cuda", on[0])
    if stream is None:
        return [torch.empty(shape, dtype=torch.int32, device=device) for shape in shapes]
    with torch.cuda.stream(torch.cuda.ExternalStream(on[1], device=device)):
        return [torch.empty(shape, dtype=torch.int32, device=device) for shape in shapes]


def _workspace(on, stream, given, need):
    """(pointer, bytes, tensor) of a workspace: the caller's, or one of `need`
    bytes allocated here."""
    if given is not None:
        return given.data_ptr(), 4 * given.numel(), given
    if need <= 0:
        return 0, 0, None
    ws, = _new(on, stream, (need + 3) // 4)
    return ws.data_ptr(), 4 * ws.numel(), ws


def _call(fn, on, *args):
    """fn(*args, stream) with the tensors' GPU current; raises on an error."""
    device, handle = on
    if torch._C._cuda_getDevice() == device:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
    if rc != MPGEMM_OK:
        raise MpgemmError(rc, fn.__name__)


def quantize_rows(X, Q, scale, order=None, top_k: int = 1, workspace=None, stream=None):
    """Rows of X to 8-bit codes: scale = max|row| / 127 and the codes nearest
    to 127 * row / max|row| (ties to even).  Returns (Q, scale).

    X (T x H): float16, bfloat16 or float32, row-major.  Q (R x H): int8,
    row-major.  scale: float32, R values.  Without ``order`` R == T; with it
    (int32, R values from :func:`route`) row p of Q is row order[p] // top_k
    of X, and rows whose order is -1 keep what they hold.  A row with an
    infinity or a NaN has a NaN scale and codes 0.  ``workspace``: a contiguous
    int32 tensor of mpgemm_rows_workspace bytes, allocated when None and of
    use."""
    if torch is None:
        _with_torch()
    _check_workspace(workspace)
    xt = _type(X, "X")
    T, H, ldx = _rows(X, "X", X.dtype)
    R, H2, ldq = _rows(Q, "Q", torch.int8)
    if H2 != H or (order is None and R != T):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, Q {tuple(Q.shape)}")
    sp = _flat(scale, "scale", torch.float32, (R,))
    op = 0 if order is None else _flat(order, "order", torch.int32, (R,))
    lib, on = load_ops(), _on(stream, X, Q, scale, order, workspace)
    wp, wb, _ws = (0, 0, None) if order is None else _workspace(
        on, stream, workspace, lib.mpgemm_rows_workspace(xt, T, H, R, int(top_k)))
    _call(lib.mpgemm_quantize_rows, on, xt, T, H, X.data_ptr(), ldx, op, R, int(top_k), Q.data_ptr(), ldq, sp, wp, wb)
    return Q, scale


def _codes(B, grouped):
    """(groups, K, N, leading dimension, group stride) of gemm_i8's B."""
    if not isinstance(B, torch.Tensor) or B.dim() != (3 if grouped else 2):
        raise ValueError("B must be 2-D, or 3-D with offsets")
    if not grouped:
        K, N = B.shape
        step, ld = B.stride()
        if step == 1 and ld >= K > 1 and N > 1 and B.dtype is torch.int8 and B.is_cuda:
            return 1, K, N, ld, 0  # the ordinary case; the rest below
        B = B.unsqueeze(0)
    G, K, N, layout, ld, stride = _matrices(B, "B", torch.int8)
    if layout != MPGEMM_COL_MAJOR:
        # one value along a dimension: the bytes lie the same in both orders
        if (K > 1 and N > 1) or (K > 1 and N == 1 and B.stride(1) != 1):
            raise ValueError("B must be column-major (unit stride along K)")
        ld = K if K > 1 else B.stride(2) if N > 1 else 1
    return G, K, N, ld, stride


def gemm_i8(A, B, C, scale_a, scale_b, bias=None, offsets=None, stream=None):
    """C <- (A @ B) * scale_a[:, None] * scale_b (+ bias), A and B 8-bit codes,
    the sum exact.  Returns C.

    A (M x K): int8, row-major.  B (K x N): int8, column-major (the transpose
    view of N x K weights).  C (M x N): float16, bfloat16 or float32,
    row-major.  scale_a: float32, M values; scale_b and bias: float32, N
    values.  With ``offsets`` (int32, groups + 1 values from :func:`route`) B
    is groups x K x N and scale_b and bias are groups x N: rows offsets[g] ..
    offsets[g+1]-1 of A and C use group g's, other rows of C keep what they
    hold."""
    if torch is None:
        _with_torch()
    ot = _type(C, "C")
    M, K, lda = _rows(A, "A", torch.int8)
    M2, N2, ldc = _rows(C, "C", C.dtype)
    G, K2, N, ldw, stride = _codes(B, offsets is not None)
    if K2 != K or M2 != M or N2 != N:
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, C {tuple(C.shape)}")
    wide = (N,) if offsets is None else (G, N)
    sa = _flat(scale_a, "scale_a", torch.float32, (M,))
    sb = _flat(scale_b, "scale_b", torch.float32, wide)
    bp = 0 if bias is None else _flat(bias, "bias", torch.float32, wide)
    op = 0 if offsets is None else _flat(offsets, "offsets", torch.int32, (G + 1,))
    _call(load_ops().mpgemm_i8_gemm, _on(stream, C, A, B, scale_a, scale_b, bias, offsets), ot, G, M, N, K,
          A.data_ptr(), lda, B.data_ptr(), ldw, stride, C.data_ptr(), ldc, sa, sb, bp, op)
    return C


def route(experts, num_experts: int, out=None, workspace=None, stream=None):
    """The order of (token, slot) pairs by expert.  Returns (order, position,
    offsets), int32.

    experts: int32 or int64, contiguous, usually T x top_k; ids outside 0 ..
    num_experts-1 are pairs without an expert.  order: the pair at each
    position of the stable sort, -1 behind the last expert's; position (of
    experts' shape): each pair's position, -1 without an expert; offsets
    (num_experts + 1): each expert's first position.
    ``out``: the three tensors to write (allocated when None).
    ``workspace``: a contiguous int32 tensor of at least
    mpgemm_route_workspace bytes; allocated when None and needed."""
    if torch is None:
        _with_torch()
    _check_workspace(workspace)
    if not isinstance(experts, torch.Tensor) or experts.dtype not in (torch.int32, torch.int64):
        raise TypeError("experts must be an int32 or int64 tensor")
    if not experts.is_cuda or not experts.is_contiguous():
        raise ValueError("experts must be contiguous, on the GPU")
    pairs, E = experts.numel(), int(num_experts)
    need = mpgemm_route_workspace(pairs, E)
    if need < 0:
        raise MpgemmError(need, "mpgemm_route")
    given = () if out is None else tuple(out)
    if out is not None and len(given) != 3:
        raise ValueError("out must be (order, position, offsets)")
    if given:
        order, position, offsets = given
        _flat(order, "order", torch.int32, (pairs,))
        _flat(position, "position", torch.int32, experts.shape)
        _flat(offsets, "offsets", torch.int32, (E + 1,))
    on = _on(stream, experts, workspace, *given)
    wp, wb, _ws = _workspace(on, stream, workspace, need)
    if not given:
        order, position, offsets = _new(on, stream, pairs, experts.shape, E + 1)
    _call(load_ops().mpgemm_route, on, MPGEMM_ID_I64 if experts.dtype == torch.int64 else MPGEMM_ID_I32, pairs, E,
          experts.data_ptr(), order.data_ptr(), position.data_ptr(), offsets.data_ptr(), wp, wb)
    return order, position, offsets


def gather_rows(X, order, Y, top_k: int = 1, workspace=None, stream=None):
    """Y[p] = X[order[p] // top_k]: tokens' rows into expert order.  Returns Y.

    X (T x H) and Y (R x H): float16, bfloat16 or float32, the same, row-major.
    order: int32, R values from :func:`route`; rows whose order is -1 keep
    what they hold.  ``workspace``: a contiguous int32 tensor of
    mpgemm_rows_workspace bytes, allocated when None and of use.  The gradient
    by X is ``combine_rows(dY, position, dX)``."""
    if torch is None:
        _with_torch()
    _check_workspace(workspace)
    ty = _type(X, "X")
    T, H, ldx = _rows(X, "X", X.dtype)
    R, H2, ldy = _rows(Y, "Y", X.dtype)
    if H2 != H:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, Y {tuple(Y.shape)}")
    op = _flat(order, "order", torch.int32, (R,))
    lib, on = load_ops(), _on(stream, Y, X, order, workspace)
    wp, wb, _ws = _workspace(on, stream, workspace, lib.mpgemm_rows_workspace(ty, T, H, R, int(top_k)))
    _call(lib.mpgemm_gather_rows, on, ty, T, H, X.data_ptr(), ldx, op, R, int(top_k), Y.data_ptr(), ldy, wp, wb)
    return Y


def _slots(position, T):
    if position.dim() != 2 or position.shape[0] != T:
        raise ValueError(f"position must be {T} x top_k, got {tuple(position.shape)}")
    return position.shape[1]


def combine_rows(Y, position, out, weights=None, stream=None):
    """out[t] = sum_s weights[t, s] * Y[position[t, s]] in FP32, slots
    ascending.  Returns out.

    Y (R x H) and out (T x H): float16, bfloat16 or float32 each, row-major.
    position: int32, T x top_k from :func:`route`; pairs at -1 add nothing.
    weights: float32, T x top_k, or None for ones."""
    if torch is None:
        _with_torch()
    yt, ot = _type(Y, "Y"), _type(out, "out")
    R, H2, ldy = _rows(Y, "Y", Y.dtype)
    T, H, ldo = _rows(out, "out", out.dtype)
    if H2 != H:
        raise ValueError(f"shape mismatch: Y {tuple(Y.shape)}, out {tuple(out.shape)}")
    pp = _flat(position, "position", torch.int32, None)
    k = _slots(position, T)
    wp = 0 if weights is None else _flat(weights, "weights", torch.float32, (T, k))
    _call(load_ops().mpgemm_combine_rows, _on(stream, out, Y, position, weights), yt, ot, T, k, H, R,
          Y.data_ptr(), ldy, pp, wp, out.data_ptr(), ldo)
    return out


def combine_rows_backward(dout, Y, position, weights, dY, dweights=None, stream=None):
    """The gradients of :func:`combine_rows`: dY[position[t, s]] = weights[t, s]
    * dout[t] and dweights[t, s] = <dout[t], Y[position[t, s]]>.  Returns
    (dY, dweights).

    dout (T x H), Y and dY (R x H): float16, bfloat16 or float32 each,
    row-major.  weights: float32, T x top_k, or None for ones.  dweights:
    float32, T x top_k, 0 for pairs at -1; None: not computed (Y may be None).
    Rows of dY that no pair has keep what they hold."""
    if torch is None:
        _with_torch()
    dt, gt = _type(dout, "dout"), _type(dY, "dY")
    T, H, ldo = _rows(dout, "dout", dout.dtype)
    R, H2, ldg = _rows(dY, "dY", dY.dtype)
    yt, ldy, yp = dt, ldo, 0
    if Y is not None:
        yt, yp = _type(Y, "Y"), Y.data_ptr()
        ldy = _rows(Y, "Y", Y.dtype)[2]
        if Y.shape != dY.shape:
            raise ValueError(f"shape mismatch: Y {tuple(Y.shape)}, dY {tuple(dY.shape)}")
    elif dweights is not None:
        raise ValueError("dweights needs Y")
    if H2 != H:
        raise ValueError(f"shape mismatch: dout {tuple(dout.shape)}, dY {tuple(dY.shape)}")
    pp = _flat(position, "position", torch.int32, None)
    k = _slots(position, T)
    wp = 0 if weights is None else _flat(weights, "weights", torch.float32, (T, k))
    gp = 0 if dweights is None else _flat(dweights, "dweights", torch.float32, (T, k))
    _call(load_ops().mpgemm_combine_rows_backward, _on(stream, dY, dout, Y, position, weights, dweights), dt, yt,
          gt, T, k, H, R, dout.data_ptr(), ldo, yp, ldy, pp, wp, dY.data_ptr(), ldg, gp)
    return dY, dweights


def gemm_grouped(A, B, C, offsets, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """C[rows of g] <- alpha * A[rows of g] @ B[g] + beta * C[rows of g] for
    every group g, its rows being offsets[g] .. offsets[g+1]-1.  Returns C.

    A (R x K, row-major) and B (groups x K x N, each row- or column-major):
    both float16 or both bfloat16.  C (R x N): float32, row-major; rows of no
    group keep what they hold.  offsets: int32, groups + 1 values.  The
    gradient by A is ``gemm_grouped(dC, B.mT, dA, offsets)``."""
    if torch is None:
        _with_torch()
    it = _type(A, "A", (MPGEMM_T_F16, MPGEMM_T_BF16))
    R, K, lda = _rows(A, "A", A.dtype)
    R2, N2, ldc = _rows(C, "C", torch.float32)
    G, K2, N, layout, ldb, stride = _matrices(B, "B", A.dtype)
    if K2 != K or R2 != R or N2 != N:
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, C {tuple(C.shape)}")
    op = _flat(offsets, "offsets", torch.int32, (G + 1,))
    _call(load_ops().mpgemm_grouped, _on(stream, C, A, B, offsets), it, layout, G, R, N, K, A.data_ptr(), lda,
          B.data_ptr(), ldb, stride, C.data_ptr(), ldc, float(alpha), float(beta), op)
    return C


def gemm_grouped_wgrad(A, B, C, offsets, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """C[g] <- alpha * A[:, rows of g] @ B[rows of g] + beta * C[g] for every
    group g: the gradient of :func:`gemm_grouped` by its weights.  Returns C.

    A (M x R, column-major: the transpose view of R x M rows) and B (R x N,
    row-major): both float16 or both bfloat16.  C (groups x M x N): float32,
    each row-major; a group without rows has beta * C[g]."""
    if torch is None:
        _with_torch()
    it = _type(A, "A", (MPGEMM_T_F16, MPGEMM_T_BF16))
    if A.dim() != 2:
        raise ValueError("A must be 2-D")
    R2, M2, lda = _rows(A.t(), "A (transposed)", A.dtype)
    R, N2, ldb = _rows(B, "B", A.dtype)
    G, M, N, layout, ldc, stride = _matrices(C, "C", torch.float32)
    if layout != MPGEMM_ROW_MAJOR:
        raise ValueError("C must be row-major")
    if M2 != M or R2 != R or N2 != N:
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, C {tuple(C.shape)}")
    op = _flat(offsets, "offsets", torch.int32, (G + 1,))
    _call(load_ops().mpgemm_grouped_wgrad, _on(stream, C, A, B, offsets), it, G, R, M, N, A.data_ptr(), lda,
          B.data_ptr(), ldb, C.data_ptr(), ldc, stride, float(alpha), float(beta), op)
    return C
