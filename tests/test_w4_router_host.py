"""Host-side tests of the 4-bit and router libraries (no GPU): the exported
symbols, the argument checks of the C ABI (before any HIP call, on fake
pointers) and of the tensor functions, workspaces, the choice of kernel, and
the generated assembly."""
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
HEADERS = {"mpgemm_w4.h": (mp.load_w4, 4), "mpgemm_router.h": (mp.load_router, 4)}


@pytest.mark.parametrize("header", list(HEADERS))
def test_library_exports_its_header_and_the_others_none_of_it(header):
    load, count = HEADERS[header]
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mpgemm_\w+)\s*\(", text)))
    assert len(names) == count
    assert not [n for n in names if not hasattr(load(), n) or not hasattr(mp, n)]
    for other in (mp.lib_path(), mp.OPS_PATH):
        assert not [n for n in names if hasattr(ctypes.CDLL(other), n)]


@pytest.mark.parametrize("header", list(HEADERS))
def test_header_compiles_as_c(header):
    src = f'#include "{header}"\nint main(void) {{ return (int)MPGEMM_T_F16; }}\n'
    res = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"),
                          "-x", "c", "-"], input=src, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def call(fn, defaults, **change):
    return fn(**{**defaults, **change})


PACK = dict(w_type=2, s_type=0, N=4, K=70, group=32, W=P, ldw=70, Q=P, ldq=35, scale=P, lds=3)
PACK_CASES = [
    (dict(w_type=3), mp.MPGEMM_ETYPE), (dict(w_type=-1), mp.MPGEMM_ETYPE), (dict(s_type=2), mp.MPGEMM_ETYPE),
    (dict(N=-1), mp.MPGEMM_EDIM), (dict(K=-1), mp.MPGEMM_EDIM), (dict(N=1 << 31), mp.MPGEMM_EDIM),
    (dict(K=(1 << 28) + 1, ldw=1 << 29, ldq=1 << 28, lds=1 << 24), mp.MPGEMM_EDIM),
    (dict(group=0), mp.MPGEMM_EDIM), (dict(group=16), mp.MPGEMM_EDIM), (dict(group=48), mp.MPGEMM_EDIM),
    (dict(group=-32), mp.MPGEMM_EDIM), (dict(group=1 << 29), mp.MPGEMM_EDIM),
    (dict(N=(1 << 31) - 1, K=4096, ldw=4096, ldq=2048, lds=128), mp.MPGEMM_EDIM),
    (dict(ldw=69), mp.MPGEMM_ELD), (dict(ldq=34), mp.MPGEMM_ELD), (dict(lds=2), mp.MPGEMM_ELD),
    (dict(K=0, ldw=0), mp.MPGEMM_ELD),
    (dict(W=0), mp.MPGEMM_ENULL), (dict(Q=0), mp.MPGEMM_ENULL), (dict(scale=0), mp.MPGEMM_ENULL),
    (dict(W=P + 2), mp.MPGEMM_EALIGN), (dict(w_type=0, W=P + 1), mp.MPGEMM_EALIGN), (dict(scale=P + 1), mp.MPGEMM_EALIGN),
    (dict(N=0, W=0, Q=0, scale=0), 0), (dict(K=0, W=0, Q=0, scale=0, ldw=1), 0),
]


@pytest.mark.parametrize("change,expect", PACK_CASES)
def test_pack_codes(change, expect):
    assert call(mp.mpgemm_w4_quantize, PACK, **change) == expect
    assert call(mp.mpgemm_w4_dequantize, PACK, **change) == expect


GEMM = dict(in_type=0, out_type=2, groups=1, M=4, N=5, K=70, group=32, A=P, lda=70, Q=P, ldq=35, stride_q=0, scale=P,
            lds=3, stride_s=0, C=P, ldc=5, bias=0, offsets=0)


@pytest.mark.parametrize("change,expect", [
    (dict(in_type=2), mp.MPGEMM_ETYPE), (dict(out_type=3), mp.MPGEMM_ETYPE), (dict(in_type=-1), mp.MPGEMM_ETYPE),
    (dict(groups=0), mp.MPGEMM_EDIM), (dict(groups=1025, offsets=P), mp.MPGEMM_EDIM), (dict(M=-1), mp.MPGEMM_EDIM),
    (dict(N=-1), mp.MPGEMM_EDIM), (dict(M=1 << 31), mp.MPGEMM_EDIM), (dict(group=33), mp.MPGEMM_EDIM),
    (dict(K=(1 << 28) + 1, lda=1 << 29, ldq=1 << 28, lds=1 << 24), mp.MPGEMM_EDIM),
    (dict(M=(1 << 31) - 1, N=(1 << 31) - 1, ldc=1 << 31), mp.MPGEMM_EDIM),
    (dict(lda=69), mp.MPGEMM_ELD), (dict(ldq=34), mp.MPGEMM_ELD), (dict(lds=2), mp.MPGEMM_ELD), (dict(ldc=4), mp.MPGEMM_ELD),
    (dict(lda=BIG), mp.MPGEMM_ELD), (dict(ldq=BIG), mp.MPGEMM_ELD), (dict(lds=BIG), mp.MPGEMM_ELD),
    (dict(stride_q=-1), mp.MPGEMM_ELD), (dict(stride_s=-1), mp.MPGEMM_ELD),
    (dict(A=0), mp.MPGEMM_ENULL), (dict(Q=0), mp.MPGEMM_ENULL), (dict(scale=0), mp.MPGEMM_ENULL), (dict(C=0), mp.MPGEMM_ENULL),
    (dict(groups=2, stride_q=175, stride_s=15), mp.MPGEMM_ENULL),
    (dict(A=P + 1), mp.MPGEMM_EALIGN), (dict(scale=P + 1), mp.MPGEMM_EALIGN), (dict(C=P + 2), mp.MPGEMM_EALIGN),
    (dict(bias=P + 2), mp.MPGEMM_EALIGN), (dict(offsets=P + 2), mp.MPGEMM_EALIGN),
    (dict(M=0, A=0, C=0), 0), (dict(N=0, Q=0, C=0, scale=0), 0),
])
def test_gemm_codes(change, expect):
    assert call(mp.mpgemm_w4_gemm, GEMM, **change) == expect


SELECT = dict(l_type=2, T=4, E=8, top_k=2, normalize=1, logits=P, ldl=8, ids=P, weights=P)


@pytest.mark.parametrize("change,expect", [
    (dict(l_type=3), mp.MPGEMM_ETYPE), (dict(T=-1), mp.MPGEMM_EDIM), (dict(T=1 << 31), mp.MPGEMM_EDIM),
    (dict(E=0, ldl=0), mp.MPGEMM_EDIM), (dict(E=1025, ldl=1025), mp.MPGEMM_EDIM), (dict(top_k=0), mp.MPGEMM_EDIM),
    (dict(top_k=9), mp.MPGEMM_EDIM), (dict(E=100, ldl=100, top_k=65), mp.MPGEMM_EDIM), (dict(ldl=7), mp.MPGEMM_ELD),
    (dict(logits=0), mp.MPGEMM_ENULL), (dict(ids=0), mp.MPGEMM_ENULL), (dict(weights=0), mp.MPGEMM_ENULL),
    (dict(logits=P + 2), mp.MPGEMM_EALIGN), (dict(l_type=0, logits=P + 1), mp.MPGEMM_EALIGN),
    (dict(ids=P + 2), mp.MPGEMM_EALIGN), (dict(weights=P + 1), mp.MPGEMM_EALIGN), (dict(T=0, logits=0, ids=0, weights=0), 0),
])
def test_select_codes(change, expect):
    assert call(mp.mpgemm_select_experts, SELECT, **change) == expect


BALANCE = dict(l_type=2, id_type=0, T=4, E=8, top_k=2, logits=P, ldl=8, ids=P, coefficient=1.0, loss=P, counts=P,
               probs=P, workspace=P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("change,expect", [
    (dict(l_type=3), mp.MPGEMM_ETYPE), (dict(id_type=2), mp.MPGEMM_ETYPE), (dict(T=-1), mp.MPGEMM_EDIM),
    (dict(E=0), mp.MPGEMM_EDIM), (dict(E=1025, ldl=1025), mp.MPGEMM_EDIM), (dict(top_k=-1), mp.MPGEMM_EDIM),
    (dict(T=1 << 20, top_k=1 << 11), mp.MPGEMM_EDIM), (dict(ldl=7), mp.MPGEMM_ELD),
    (dict(logits=0), mp.MPGEMM_ENULL), (dict(ids=0), mp.MPGEMM_ENULL), (dict(loss=0), mp.MPGEMM_ENULL),
    (dict(counts=0), mp.MPGEMM_ENULL), (dict(workspace=0), mp.MPGEMM_ENULL),
    (dict(logits=P + 2), mp.MPGEMM_EALIGN), (dict(id_type=1, ids=P + 4), mp.MPGEMM_EALIGN), (dict(ids=P + 2), mp.MPGEMM_EALIGN),
    (dict(loss=P + 2), mp.MPGEMM_EALIGN), (dict(counts=P + 1), mp.MPGEMM_EALIGN), (dict(probs=P + 2), mp.MPGEMM_EALIGN),
    (dict(workspace=P + 2), mp.MPGEMM_EALIGN), (dict(workspace_bytes=16), mp.MPGEMM_EWORKSPACE),
])
def test_balance_codes(change, expect):
    assert call(mp.mpgemm_balance_loss, BALANCE, **change) == expect


@pytest.mark.parametrize("T,E,k", [(0, 1, 0), (1, 1, 1), (64, 8, 2), (65, 8, 2), (1 << 20, 1024, 8), ((1 << 31) - 1, 256, 1)])
def test_balance_workspace(T, E, k):
    need = mp.mpgemm_balance_workspace(T, E, k)
    assert need % 4 == 0 and 0 < need <= 4 * (512 * (2 * E + 1) + 1 + 3 * (E // 16 + 1))
    # one byte less is refused, before any pointer is looked at twice
    assert call(mp.mpgemm_balance_loss, BALANCE, T=T, E=E, top_k=k, ldl=E, workspace_bytes=need - 1) == mp.MPGEMM_EWORKSPACE


@pytest.mark.parametrize("T,E,k", [(-1, 8, 1), (8, 0, 1), (8, 1025, 1), (8, 8, -1), (1 << 31, 8, 1), (1 << 30, 8, 2)])
def test_balance_workspace_refuses(T, E, k):
    assert mp.mpgemm_balance_workspace(T, E, k) == mp.MPGEMM_EDIM


BACK = dict(l_type=2, d_type=1, id_type=0, T=4, E=8, top_k=2, normalize=1, logits=P, ldl=8, ids=P, dweights=P, counts=P,
            coefficient=1.0, dloss=P, dlogits=P, ldd=8)


@pytest.mark.parametrize("change,expect", [
    (dict(l_type=3), mp.MPGEMM_ETYPE), (dict(d_type=3), mp.MPGEMM_ETYPE), (dict(id_type=2), mp.MPGEMM_ETYPE),
    (dict(T=-1), mp.MPGEMM_EDIM), (dict(E=0, ldl=8), mp.MPGEMM_EDIM), (dict(top_k=65), mp.MPGEMM_EDIM),
    (dict(top_k=-1), mp.MPGEMM_EDIM), (dict(ldl=7), mp.MPGEMM_ELD), (dict(ldd=7), mp.MPGEMM_ELD),
    (dict(logits=0), mp.MPGEMM_ENULL), (dict(dlogits=0), mp.MPGEMM_ENULL), (dict(ids=0), mp.MPGEMM_ENULL),
    (dict(logits=P + 2), mp.MPGEMM_EALIGN), (dict(dlogits=P + 1), mp.MPGEMM_EALIGN), (dict(ids=P + 2), mp.MPGEMM_EALIGN),
    (dict(id_type=1, ids=P + 4), mp.MPGEMM_EALIGN), (dict(dweights=P + 2), mp.MPGEMM_EALIGN),
    (dict(counts=P + 2), mp.MPGEMM_EALIGN), (dict(dloss=P + 1), mp.MPGEMM_EALIGN),
    (dict(T=0, logits=0, dlogits=0, ids=0), 0),
])
def test_backward_codes(change, expect):
    assert call(mp.mpgemm_router_backward, BACK, **change) == expect


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


H, U8, I32 = torch.float16, torch.uint8, torch.int32


@pytest.mark.parametrize("fn,args,kwargs,error", [
    (mp.quantize_w4, (t(2, 64, dtype=torch.float64), t(2, 32, dtype=U8), t(2, 2, dtype=H)), {}, TypeError),
    (mp.quantize_w4, (t(2, 64), t(2, 32, dtype=U8), t(2, 2, dtype=H)), {}, ValueError),            # not on the GPU
    (mp.quantize_w4, (t(2, 64), t(2, 32, dtype=U8), t(2, 2, dtype=H)), {"group": 0}, ValueError),
    (mp.dequantize_w4, (t(2, 32, dtype=U8), t(2, 2, dtype=H), t(2, 64, dtype=I32)), {}, TypeError),
    (mp.gemm_w4, (t(2, 64), t(2, 32, dtype=U8), t(2, 1, dtype=H), t(2, 2)), {}, TypeError),        # FP32 tokens
    (mp.gemm_w4, (t(2, 64, dtype=H), t(2, 32, dtype=U8), t(2, 1, dtype=H), t(2, 2, dtype=I32)), {}, TypeError),
    (mp.select_experts, (t(2, 8, dtype=I32), t(2, 2, dtype=I32), t(2, 2)), {}, TypeError),
    (mp.select_experts, (t(2, 8), t(2, 2, dtype=I32), t(2, 2)), {}, ValueError),
    (mp.balance_loss, (t(2, 8, dtype=I32), t(2, 2, dtype=I32), t(1), t(9, dtype=I32)), {}, TypeError),
    (mp.balance_loss, (t(2, 8), t(2, 2, dtype=I32), t(1), t(9, dtype=I32)), {"workspace": t(4)}, TypeError),
    (mp.router_backward, (t(2, 8), None, t(2, 8, dtype=I32)), {}, (TypeError, ValueError)),
])
def test_tensor_checks(fn, args, kwargs, error):
    with pytest.raises(error):
        fn(*args, **kwargs)


def test_query_reports_each_choice_and_refuses_what_the_product_refuses():
    assert mp.mpgemm_w4_query(0, 0, 8, 64, 32, 64, 32, 2) == dict.fromkeys(
        ("narrow", "bm", "bn", "bk", "stages", "waves", "workgroups"), 0)
    seen = set()
    for M in (1, 4, 5, 8, 16, 17, 33, 65, 129, 300, 1000, 5000):
        for N in (1, 500, 4096, 7000, 9000, 40000):
            for K in (1, 127, 128, 2000, 8192):
                k = mp.mpgemm_w4_query(0, M, N, K, 64, K, (K + 1) // 2, -(-K // 64))
                seen.add((k["narrow"], k["bm"], k["bn"], k["waves"]))
                assert k["workgroups"] == -(-M // k["bm"]) * -(-N // k["bn"])
                assert k["narrow"] or K >= 128
    assert len(seen) == 11
    with pytest.raises(mp.MpgemmError):
        mp.mpgemm_w4_query(0, 4, 4, 64, 48, 64, 32, 2)


@pytest.fixture(scope="module", params=["W4_SRC", "ROUTER_SRC"])
def device_asm(request, tmp_path_factory):
    if shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("isa") / "lib.s"
    flags = [f for f in mpbuild.flags() if f not in ("-shared", "-fPIC")]
    res = subprocess.run([mpbuild.hipcc(), *flags, "--cuda-device-only", "-S", getattr(mpbuild, request.param), "-o",
                          str(out)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    return request.param, out.read_text()


def test_generated_code(device_asm):
    """M0 is only written by the copy sequence (see test_isa_guard); nothing goes
    to scratch, whose accesses the copies' waits do not count; no packed FP32."""
    which, text = device_asm
    ins = [s for s in (line.split(";")[0].strip() for line in text.splitlines())
           if s and not s.endswith(":") and not s.startswith(".")]
    uses = [i for i, s in enumerate(ins) if re.search(r"\bm0\b", s)]
    assert bool(uses) == (which == "W4_SRC")
    for i in uses:
        assert re.fullmatch(r"s_mov_b32 m0, s\d+", ins[i]), ins[i]
        assert ins[i + 1] == "s_nop 0" and ins[i + 2].startswith("buffer_load_dword") and ins[i + 2].endswith(" lds")
    kernels = re.findall(r"\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", text, re.S)
    assert len(kernels) > 50
    for name, body in kernels:
        assert int(re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", body).group(1)) == 0, name
    assert not re.findall(r"\bv_pk_(?:add|mul|fma)_f32\b", text)
