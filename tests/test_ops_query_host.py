"""Host-side tests of the operator library's queries (no GPU): the exported
symbols, argument checks, and that the sizes of the GPU tests take the kernels
they are meant for."""
import ctypes
import os
import re
import subprocess

import pytest

import dense_mixed_precision_amd as mp
from tests import ops_kernels as ok
from tests.test_ops_host import ROOT, call

HEADER = os.path.join(ROOT, "include", "mpgemm_ops_query.h")
BIG = 1 << 40


def test_library_exports_its_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(mpgemm_\w+)\s*\(", text))
    assert names == {"mpgemm_i8_query", "mpgemm_grouped_query", "mpgemm_grouped_wgrad_query"}
    lib = mp.load_ops()
    assert all(hasattr(lib, n) and hasattr(mp, n) for n in names)
    src = '#include "mpgemm_ops_query.h"\nint main(void) { return sizeof(mpgemm_ops_kernel) == 32 ? 0 : 1; }\n'
    res = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"),
                          "-x", "c", "-"], input=src, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


I8 = dict(groups=0, M=4, N=4, K=8, lda=8, ldw=8)
GROUPED = dict(layout_b=0, groups=2, R=4, N=8, K=8, lda=8, ldb=8, ldc=8)
WGRAD = dict(groups=2, R=4, M=8, N=8, lda=8, ldb=8, ldc=8)


@pytest.mark.parametrize("fn,defaults,change,code", [
    (mp.mpgemm_i8_query, I8, dict(groups=-1), mp.MPGEMM_EDIM), (mp.mpgemm_i8_query, I8, dict(groups=1025), mp.MPGEMM_EDIM),
    (mp.mpgemm_i8_query, I8, dict(K=131072, lda=BIG, ldw=BIG), mp.MPGEMM_EDIM),
    (mp.mpgemm_i8_query, I8, dict(lda=7), mp.MPGEMM_ELD), (mp.mpgemm_i8_query, I8, dict(ldw=BIG), mp.MPGEMM_ELD),
    (mp.mpgemm_i8_query, I8, dict(M=(1 << 31) - 1, N=(1 << 31) - 1), mp.MPGEMM_EDIM),
    (mp.mpgemm_grouped_query, GROUPED, dict(layout_b=2), mp.MPGEMM_ELAYOUT),
    (mp.mpgemm_grouped_query, GROUPED, dict(groups=0), mp.MPGEMM_EDIM),
    (mp.mpgemm_grouped_query, GROUPED, dict(ldc=7), mp.MPGEMM_ELD),
    (mp.mpgemm_grouped_query, GROUPED, dict(ldb=BIG), mp.MPGEMM_ELD),
    (mp.mpgemm_grouped_wgrad_query, WGRAD, dict(R=-1), mp.MPGEMM_EDIM),
    (mp.mpgemm_grouped_wgrad_query, WGRAD, dict(lda=7), mp.MPGEMM_ELD),
    (mp.mpgemm_grouped_wgrad_query, WGRAD, dict(ldb=BIG), mp.MPGEMM_ELD),
])
def test_refusals(fn, defaults, change, code):
    with pytest.raises(mp.MpgemmError) as e:
        call(fn, defaults, **change)
    assert e.value.code == code


def test_no_place_for_the_answer_and_nothing_to_launch():
    lib, none = mp.load_ops(), ctypes.POINTER(mp._ops.MpgemmOpsKernel)()
    assert lib.mpgemm_i8_query(0, 4, 4, 8, 8, 8, none) == mp.MPGEMM_ENULL
    assert lib.mpgemm_grouped_query(0, 2, 4, 8, 8, 8, 8, 8, none) == mp.MPGEMM_ENULL
    assert lib.mpgemm_grouped_wgrad_query(2, 4, 8, 8, 8, 8, 8, none) == mp.MPGEMM_ENULL
    for answer in (call(mp.mpgemm_i8_query, I8, M=0), call(mp.mpgemm_grouped_query, GROUPED, N=0),
                   call(mp.mpgemm_grouped_wgrad_query, WGRAD, M=0)):
        assert not any(answer.values())


def test_workgroups():
    """One for each tile of any split of the rows."""
    assert mp.mpgemm_i8_query(0, 8, 8192, 8192, 8192, 8192) == dict(narrow=1, bm=16, bn=16, bk=0, stages=0, waves=8,
                                                                   workgroups=512)
    big = mp.mpgemm_grouped_query(1, 32, 32768, 2048, 2048, 2048, 2048, 2048)
    assert big == dict(narrow=0, bm=256, bn=256, bk=64, stages=2, waves=8, workgroups=(32768 + 32 * 255) // 256 * 8)
    assert mp.mpgemm_grouped_wgrad_query(32, 32768, 2048, 2048, 2048, 2048, 2048)["workgroups"] == 32 * 64


@pytest.mark.parametrize("gap", [0, 5])
def test_sizes_take_their_kernels(gap):
    for kernel, (M, N, Ks) in ok.I8.items():
        assert [ok.i8_kernel(0, M, N, K, gap) for K in Ks] == [kernel] * len(Ks)
    for kernel, (G, M, N, Ks) in ok.I8_GROUPS.items():
        assert [ok.i8_kernel(G, M, N, K, gap) for K in Ks] == [kernel] * len(Ks)
    for (kernel, lb), (G, R, N, Ks) in ok.GROUPED.items():
        assert [ok.grouped_kernel(lb, G, R, N, K, gap) for K in Ks] == [kernel] * len(Ks)
    for kernel, (G, R, M, N) in ok.WGRAD.items():
        assert ok.wgrad_kernel(G, R, M, N, gap) == kernel


def test_every_kernel_has_its_sizes():
    """No table entry of the library without sizes above: the entries as the
    source lists them."""
    src = open(os.path.join(ROOT, "dense_mixed_precision_amd", "csrc", "ops.hip")).read()
    tiles = {tuple(map(int, m)) for m in re.findall(r"I8Cfg<(\d+), (\d+), (\d+), \d+, \d+, (\d+)>", src)}
    assert {f"{m}x{n}x{k}, {s} stages" for m, n, k, s in tiles} == {k for k in ok.I8 if "x" in k}
    assert set(ok.I8) == set(ok.I8_GROUPS)

    def entries(table):
        body = src[src.index(f"*{table}_table()"):]
        body = body[:body.index("return table;")]
        return {f"{m}x{n}x{k}, {s} stages" for m, n, k, s in
                re.findall(r"PipeCfg<(\d+), (\d+), (\d+), \d+, \d+, (\d+),", body)}

    for lb in (ok.ROW, ok.COL):
        assert entries("rows") == {k for k, b in ok.GROUPED if b == lb and "x" in k}
    assert entries("wgrad") == set(ok.WGRAD)
