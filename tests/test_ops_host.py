"""Host-side tests of the operator library (no GPU): the exported symbols, the
argument checks of the C ABI (before any HIP call, on fake pointers) and of
the tensor functions, the workspace plan, and the generated assembly."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import dense_mixed_precision_amd as mp
from dense_mixed_precision_amd import build as mpbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x7F0000000000  # a 256-byte aligned fake device address
BIG = 1 << 40


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mpgemm_ops.h")).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(mpgemm_\w+)\s*\(", text)))


def test_library_exports_its_header_and_the_gemm_library_none_of_it():
    names = declared()
    assert len(names) == 10
    lib = mp.load_ops()
    assert not [n for n in names if not hasattr(lib, n)]
    product = ctypes.CDLL(mp.lib_path())
    assert not [n for n in names if hasattr(product, n)]
    assert not [n for n in names if not hasattr(mp, n)]


def test_header_compiles_as_c():
    src = '#include "mpgemm_ops.h"\nint main(void) { return (int)MPGEMM_T_F16; }\n'
    res = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"),
                          "-x", "c", "-"], input=src, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def call(fn, defaults, **change):
    return fn(**{**defaults, **change})


QUANT = dict(x_type=0, T=4, H=8, X=P, ldx=8, order=0, R=4, top_k=1, Q=P, ldq=8, scale=P)


@pytest.mark.parametrize("change,expect", [
    (dict(x_type=3), mp.MPGEMM_ETYPE), (dict(x_type=-1), mp.MPGEMM_ETYPE),
    (dict(T=-1), mp.MPGEMM_EDIM), (dict(H=-1), mp.MPGEMM_EDIM), (dict(R=3), mp.MPGEMM_EDIM),
    (dict(T=1 << 31, R=1 << 31), mp.MPGEMM_EDIM), (dict(order=P, top_k=0), mp.MPGEMM_EDIM),
    (dict(H=(1 << 28) + 1, ldx=1 << 30, ldq=1 << 30), mp.MPGEMM_EDIM),
    (dict(ldx=7), mp.MPGEMM_ELD), (dict(ldq=7), mp.MPGEMM_ELD), (dict(H=0, ldx=0), mp.MPGEMM_ELD),
    (dict(X=0), mp.MPGEMM_ENULL), (dict(Q=0), mp.MPGEMM_ENULL), (dict(scale=0), mp.MPGEMM_ENULL),
    (dict(X=P + 1), mp.MPGEMM_EALIGN), (dict(x_type=2, X=P + 2), mp.MPGEMM_EALIGN),
    (dict(order=P + 2), mp.MPGEMM_EALIGN), (dict(scale=P + 2), mp.MPGEMM_EALIGN),
    (dict(T=0, R=0, X=0, Q=0, scale=0), 0), (dict(order=P, R=0, Q=0, scale=0), 0), (dict(order=P, workspace=P + 2), mp.MPGEMM_EALIGN),
])
def test_quantize_codes(change, expect):
    assert call(mp.mpgemm_quantize_rows, QUANT, **change) == expect


I8 = dict(out_type=2, groups=1, M=4, N=4, K=8, A=P, lda=8, W=P, ldw=8, stride_w=0, C=P, ldc=4, scale_a=P, scale_w=P,
          bias=0, offsets=0)


@pytest.mark.parametrize("change,expect", [
    (dict(out_type=3), mp.MPGEMM_ETYPE),
    (dict(groups=0), mp.MPGEMM_EDIM), (dict(groups=1025, offsets=P), mp.MPGEMM_EDIM),
    (dict(M=-1), mp.MPGEMM_EDIM), (dict(N=-1), mp.MPGEMM_EDIM), (dict(K=-1), mp.MPGEMM_EDIM),
    (dict(K=131072, lda=131072, ldw=131072), mp.MPGEMM_EDIM), (dict(M=1 << 31), mp.MPGEMM_EDIM),
    (dict(lda=7), mp.MPGEMM_ELD), (dict(ldw=7), mp.MPGEMM_ELD), (dict(ldc=3), mp.MPGEMM_ELD),
    (dict(stride_w=-8), mp.MPGEMM_ELD), (dict(lda=BIG), mp.MPGEMM_ELD), (dict(ldw=BIG), mp.MPGEMM_ELD),
    (dict(ldw=1 << 62), mp.MPGEMM_ELD),
    (dict(A=0), mp.MPGEMM_ENULL), (dict(W=0), mp.MPGEMM_ENULL), (dict(C=0), mp.MPGEMM_ENULL),
    (dict(scale_a=0), mp.MPGEMM_ENULL), (dict(scale_w=0), mp.MPGEMM_ENULL),
    (dict(groups=2, stride_w=32), mp.MPGEMM_ENULL),
    (dict(C=P + 2), mp.MPGEMM_EALIGN), (dict(out_type=0, C=P + 1), mp.MPGEMM_EALIGN),
    (dict(scale_a=P + 1), mp.MPGEMM_EALIGN), (dict(bias=P + 2), mp.MPGEMM_EALIGN),
    (dict(offsets=P + 2), mp.MPGEMM_EALIGN),
    (dict(M=0, A=0, C=0), 0), (dict(N=0, W=0, C=0), 0),
    # a grid that no launch holds
    (dict(M=(1 << 31) - 1, N=(1 << 31) - 1, ldc=1 << 31), mp.MPGEMM_EDIM),
])
def test_i8_codes(change, expect):
    assert call(mp.mpgemm_i8_gemm, I8, **change) == expect


ROUTE = dict(id_type=0, pairs=8, experts=4, ids=P, order=P, position=P, offsets=P)


@pytest.mark.parametrize("change,expect", [
    (dict(id_type=2), mp.MPGEMM_ETYPE), (dict(pairs=-1), mp.MPGEMM_EDIM), (dict(pairs=(1 << 30) + 1), mp.MPGEMM_EDIM),
    (dict(experts=0), mp.MPGEMM_EDIM), (dict(experts=1025), mp.MPGEMM_EDIM),
    (dict(ids=0), mp.MPGEMM_ENULL), (dict(order=0), mp.MPGEMM_ENULL), (dict(position=0), mp.MPGEMM_ENULL),
    (dict(offsets=0), mp.MPGEMM_ENULL), (dict(pairs=0, offsets=0), mp.MPGEMM_ENULL),
    (dict(ids=P + 2), mp.MPGEMM_EALIGN), (dict(id_type=1, ids=P + 4), mp.MPGEMM_EALIGN),
    (dict(order=P + 1), mp.MPGEMM_EALIGN), (dict(workspace=P + 2, workspace_bytes=64), mp.MPGEMM_EALIGN),
    (dict(pairs=1 << 20), mp.MPGEMM_ENULL),
    (dict(pairs=1 << 20, workspace=P, workspace_bytes=64), mp.MPGEMM_EWORKSPACE),
])
def test_route_codes(change, expect):
    assert call(mp.mpgemm_route, ROUTE, **change) == expect


@pytest.mark.parametrize("pairs", [0, 1, 63, 64, 4096, 4097, 10000, 131072, 1 << 20, (1 << 30) - 1, 1 << 30])
@pytest.mark.parametrize("experts", [1, 8, 128, 1024])
def test_route_workspace(pairs, experts):
    need = mp.mpgemm_route_workspace(pairs, experts)
    assert need % (4 * (experts + 1)) == 0
    blocks = need // (4 * (experts + 1))
    assert (blocks == 0) == (pairs <= 4096) and blocks <= 256


GATHER = dict(type_=0, T=4, H=8, X=P, ldx=8, order=P, R=8, top_k=2, Y=P, ldy=8)


@pytest.mark.parametrize("change,expect", [
    (dict(type_=3), mp.MPGEMM_ETYPE), (dict(T=-1), mp.MPGEMM_EDIM), (dict(top_k=0), mp.MPGEMM_EDIM),
    (dict(R=1 << 31), mp.MPGEMM_EDIM), (dict(ldx=7), mp.MPGEMM_ELD), (dict(ldy=7), mp.MPGEMM_ELD),
    (dict(X=0), mp.MPGEMM_ENULL), (dict(Y=0), mp.MPGEMM_ENULL), (dict(order=0), mp.MPGEMM_ENULL),
    (dict(X=P + 1), mp.MPGEMM_EALIGN), (dict(type_=2, Y=P + 2), mp.MPGEMM_EALIGN), (dict(order=P + 2), mp.MPGEMM_EALIGN),
    (dict(R=0, Y=0), 0), (dict(H=0, X=0, Y=0), 0), (dict(workspace=P + 1), mp.MPGEMM_EALIGN),
])
def test_gather_codes(change, expect):
    assert call(mp.mpgemm_gather_rows, GATHER, **change) == expect


@pytest.mark.parametrize("type_,T,H,R,top_k,expect", [
    (1, 16384, 2048, 131072, 8, 4 * 131072),        # 512 MiB of rows
    (1, 16384, 2048, 131072, 1, 0),                 # every token once
    (1, 64, 2048, 256, 4, 0),                       # few rows
    (1, 16384, 2048, 16384, 8, 0),                  # most pairs have no row
    (3, 1, 1, 1, 1, mp.MPGEMM_ETYPE), (0, -1, 1, 1, 1, mp.MPGEMM_EDIM), (0, 1, 1, 1, 0, mp.MPGEMM_EDIM),
    (2, (1 << 31) - 1, 1 << 28, (1 << 31) - 1, (1 << 31) - 1, 0), (0, 1, (1 << 28) + 1, 1, 1, mp.MPGEMM_EDIM),
])
def test_rows_workspace(type_, T, H, R, top_k, expect):
    assert mp.mpgemm_rows_workspace(type_, T, H, R, top_k) == expect


COMBINE = dict(y_type=2, o_type=1, T=4, top_k=2, H=8, R=8, Y=P, ldy=8, position=P, weights=P, O=P, ldo=8)


@pytest.mark.parametrize("change,expect", [
    (dict(y_type=3), mp.MPGEMM_ETYPE), (dict(o_type=-1), mp.MPGEMM_ETYPE), (dict(T=-1), mp.MPGEMM_EDIM),
    (dict(top_k=-1), mp.MPGEMM_EDIM), (dict(ldy=7), mp.MPGEMM_ELD), (dict(ldo=7), mp.MPGEMM_ELD),
    (dict(Y=0), mp.MPGEMM_ENULL), (dict(O=0), mp.MPGEMM_ENULL), (dict(position=0), mp.MPGEMM_ENULL),
    (dict(Y=P + 2), mp.MPGEMM_EALIGN), (dict(O=P + 1), mp.MPGEMM_EALIGN), (dict(weights=P + 2), mp.MPGEMM_EALIGN),
    (dict(T=0, O=0), 0), (dict(H=0, O=0), 0),
])
def test_combine_codes(change, expect):
    assert call(mp.mpgemm_combine_rows, COMBINE, **change) == expect


BACK = dict(d_type=1, y_type=2, dy_type=1, T=4, top_k=2, H=8, R=8, dO=P, ldo=8, Y=P, ldy=8, position=P, weights=P,
            dY=P, lddy=8, dweights=P)


@pytest.mark.parametrize("change,expect", [
    (dict(d_type=3), mp.MPGEMM_ETYPE), (dict(y_type=3), mp.MPGEMM_ETYPE), (dict(dy_type=3), mp.MPGEMM_ETYPE),
    (dict(T=-1), mp.MPGEMM_EDIM), (dict(T=1 << 30, top_k=8), mp.MPGEMM_EDIM),
    (dict(ldo=7), mp.MPGEMM_ELD), (dict(ldy=7), mp.MPGEMM_ELD), (dict(lddy=7), mp.MPGEMM_ELD),
    (dict(dO=0), mp.MPGEMM_ENULL), (dict(Y=0), mp.MPGEMM_ENULL), (dict(dY=0), mp.MPGEMM_ENULL),
    (dict(position=0), mp.MPGEMM_ENULL), (dict(Y=P + 2), mp.MPGEMM_EALIGN), (dict(dweights=P + 2), mp.MPGEMM_EALIGN),
    (dict(T=0, dO=0, dY=0), 0), (dict(top_k=0, position=0), 0),
])
def test_combine_backward_codes(change, expect):
    assert call(mp.mpgemm_combine_rows_backward, BACK, **change) == expect


GROUPED = dict(in_type=0, layout_b=0, groups=2, R=4, N=8, K=8, A=P, lda=8, B=P, ldb=8, stride_b=64, C=P, ldc=8,
               alpha=1.0, beta=0.0, offsets=P)


@pytest.mark.parametrize("change,expect", [
    (dict(in_type=2), mp.MPGEMM_ETYPE), (dict(layout_b=2), mp.MPGEMM_ELAYOUT),
    (dict(groups=0), mp.MPGEMM_EDIM), (dict(groups=1025), mp.MPGEMM_EDIM), (dict(R=-1), mp.MPGEMM_EDIM),
    (dict(K=1 << 31, lda=1 << 31), mp.MPGEMM_EDIM),
    (dict(lda=7), mp.MPGEMM_ELD), (dict(ldb=7), mp.MPGEMM_ELD), (dict(layout_b=1, K=9, lda=9), mp.MPGEMM_ELD),
    (dict(ldc=7), mp.MPGEMM_ELD), (dict(stride_b=-1), mp.MPGEMM_ELD), (dict(lda=BIG), mp.MPGEMM_ELD),
    (dict(ldb=BIG), mp.MPGEMM_ELD), (dict(ldc=1 << 62), mp.MPGEMM_ELD),
    (dict(A=0), mp.MPGEMM_ENULL), (dict(B=0), mp.MPGEMM_ENULL), (dict(C=0), mp.MPGEMM_ENULL),
    (dict(offsets=0), mp.MPGEMM_ENULL),
    (dict(A=P + 1), mp.MPGEMM_EALIGN), (dict(C=P + 2), mp.MPGEMM_EALIGN), (dict(offsets=P + 2), mp.MPGEMM_EALIGN),
    (dict(R=0, A=0, C=0), 0), (dict(N=0, B=0, C=0), 0),
])
def test_grouped_codes(change, expect):
    assert call(mp.mpgemm_grouped, GROUPED, **change) == expect


WGRAD = dict(in_type=0, groups=2, R=4, M=8, N=8, A=P, lda=8, B=P, ldb=8, C=P, ldc=8, stride_c=64, alpha=1.0,
             beta=0.0, offsets=P)


@pytest.mark.parametrize("change,expect", [
    (dict(in_type=2), mp.MPGEMM_ETYPE), (dict(groups=0), mp.MPGEMM_EDIM), (dict(M=-1), mp.MPGEMM_EDIM),
    (dict(lda=7), mp.MPGEMM_ELD), (dict(ldb=7), mp.MPGEMM_ELD), (dict(ldc=7), mp.MPGEMM_ELD),
    (dict(stride_c=63), mp.MPGEMM_ELD), (dict(stride_c=-64), mp.MPGEMM_ELD), (dict(ldb=BIG), mp.MPGEMM_ELD),
    (dict(A=0), mp.MPGEMM_ENULL), (dict(B=0), mp.MPGEMM_ENULL), (dict(C=0), mp.MPGEMM_ENULL),
    (dict(offsets=0), mp.MPGEMM_ENULL), (dict(B=P + 1), mp.MPGEMM_EALIGN), (dict(C=P + 2), mp.MPGEMM_EALIGN),
    (dict(M=0, C=0), 0), (dict(N=0, C=0), 0),
])
def test_wgrad_codes(change, expect):
    assert call(mp.mpgemm_grouped_wgrad, WGRAD, **change) == expect


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("fn,args,error", [
    (mp.quantize_rows, (t(2, 4, dtype=torch.float64), t(2, 4, dtype=torch.int8), t(2)), TypeError),
    (mp.quantize_rows, (t(2, 4), t(2, 4), t(2)), ValueError),                     # not on the GPU
    (mp.gemm_i8, (t(2, 4, dtype=torch.float16), t(4, 2), t(2, 2), t(2), t(2)), TypeError),
    (mp.gemm_i8, (t(2, 4, dtype=torch.int8), t(4, 2), t(2, 2, dtype=torch.int8), t(2), t(2)), TypeError),
    (mp.route, (t(2, 2), 4), TypeError),
    (mp.route, (t(2, 2, dtype=torch.int32), 4), ValueError),
    (mp.gather_rows, (t(2, 4, dtype=torch.int32), t(2), t(2, 4)), TypeError),
    (mp.combine_rows, ([], t(2), t(2, 4)), TypeError),
    (mp.combine_rows_backward, (t(2, 4), None, t(2), None, t(2, 4, dtype=torch.int8)), TypeError),
    (mp.gemm_grouped, (t(2, 4), t(2, 4, 4), t(2, 4), t(3)), TypeError),
    (mp.gemm_grouped_wgrad, (t(2, 4), t(2, 4), t(2, 4, 4), t(3)), TypeError),
])
def test_tensor_checks(fn, args, error):
    with pytest.raises(error):
        fn(*args)


@pytest.mark.parametrize("workspace", ["no tensor", [0, 0], t(8), t(8, 2, dtype=torch.int32).t()])
@pytest.mark.parametrize("fn,args", [
    (mp.quantize_rows, (t(2, 4), t(2, 4, dtype=torch.int8), t(2))),
    (mp.route, (t(2, 2, dtype=torch.int32), 4)),
    (mp.gather_rows, (t(2, 4), t(2, dtype=torch.int32), t(2, 4))),
])
def test_workspace_is_checked_first(fn, args, workspace):
    with pytest.raises(TypeError, match="workspace"):
        fn(*args, workspace=workspace)


@pytest.fixture(scope="module")
def device_asm(tmp_path_factory):
    if shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("isa") / "ops.s"
    flags = [f for f in mpbuild.flags() if f not in ("-shared", "-fPIC")]
    cmd = [mpbuild.hipcc(), *flags, "--cuda-device-only", "-S", mpbuild.OPS_SRC, "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    return out.read_text()


def test_m0_is_only_written_by_the_copy_sequence(device_asm):
    """The LDS copies set M0 behind the compiler's back, so nothing else in
    those kernels may use it (see test_isa_guard)."""
    ins = [s for s in (line.split(";")[0].strip() for line in device_asm.splitlines())
           if s and not s.endswith(":") and not s.startswith(".")]
    uses = [i for i, s in enumerate(ins) if re.search(r"\bm0\b", s)]
    assert uses
    for i in uses:
        assert re.fullmatch(r"s_mov_b32 m0, s\d+", ins[i]), ins[i]
        assert ins[i + 1] == "s_nop 0" and ins[i + 2].startswith("buffer_load_dword") and ins[i + 2].endswith(" lds")


def test_no_private_scratch_and_no_packed_fp32(device_asm):
    kernels = re.findall(r"\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", device_asm, re.S)
    assert any("i8_tile" in n for n, _ in kernels) and any("gemm_grouped_pipe" in n for n, _ in kernels)
    for name, body in kernels:
        assert int(re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", body).group(1)) == 0, name
    assert not re.findall(r"\bv_pk_(?:add|mul|fma)_f32\b", device_asm)
