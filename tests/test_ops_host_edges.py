"""Host-side tests of the operator library at its edges (no GPU): slots a
token beyond what the kernels' counters hold, the widest rows, first calls on
several threads, arithmetic that no compiler option may change."""
import os
import re
import shutil
import subprocess
import sys

import pytest

import dense_mixed_precision_amd as mp
from dense_mixed_precision_amd import _ops
from dense_mixed_precision_amd import build as mpbuild
from tests.test_ops_host import BACK, COMBINE, GATHER, QUANT, ROOT, call

MOST = 1 << 30  # slots a token; mpgemm_route makes no more pairs


@pytest.mark.parametrize("top_k,expect", [(MOST, 0), (MOST + 1, mp.MPGEMM_EDIM), ((1 << 31) - 1, mp.MPGEMM_EDIM)])
def test_combine_limits_the_slots(top_k, expect):
    """The kernel walks the slots four at a time in 32 bits: just below 2^31
    its counter would wrap and never reach the end."""
    assert call(mp.mpgemm_combine_rows, COMBINE, T=0, top_k=top_k) == expect


def test_way_by_tokens_limits_the_slots():
    """One token with about 2^31 slots: eight at a time wrap a 32-bit counter,
    so its rows are made one by one, without a workspace."""
    rows = (1 << 31) - 1
    assert mp.mpgemm_rows_workspace(mp.MPGEMM_T_F16, 1, 4096, rows, MOST) == 4 * MOST
    assert mp.mpgemm_rows_workspace(mp.MPGEMM_T_F16, 1, 4096, rows, MOST + 1) == 0
    assert mp.mpgemm_rows_workspace(mp.MPGEMM_T_F16, 1, 4096, rows, rows) == 0


def test_first_call_publishes_nothing_half_made(monkeypatch):
    """Entry points test `torch is None` alone: whatever line of the first
    call's preparation another thread comes in at, torch is there only with
    the table of its types complete."""
    monkeypatch.setattr(_ops, "torch", None)
    monkeypatch.setattr(_ops, "_TYPES", {})
    seen = []

    def trace(frame, event, arg):
        if frame.f_code is not _ops._with_torch.__code__:
            return None
        seen.append((_ops.torch is not None, len(_ops._TYPES)))
        return trace

    before = sys.gettrace()
    sys.settrace(trace)
    try:
        _ops._with_torch()
    finally:
        sys.settrace(before)
    assert seen[0] == (False, 0) and seen[-1] == (True, 3)
    assert all(types == 3 for there, types in seen if there)


@pytest.mark.parametrize("contract", ["off", "on", "fast"])
def test_scales_and_bias_are_one_arithmetic(contract, tmp_path):
    """The last scale and the bias of the 8-bit product round once, as the
    header states, whether or not the compiler contracts products and sums."""
    if shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("hipcc not available")
    src, out = tmp_path / "value.hip", tmp_path / "value.s"
    src.write_text("""
#include <hip/hip_runtime.h>
#include <stdint.h>
#define MPGEMM_GROUPED
#include "kernels.hpp"
namespace mpg {
#include "i8_kernels.hpp"
__global__ void value(const int *s, const float *a, float *out) { *out = i8_value(*s, a[0], a[1], a[2], true); }
}
""")
    flags = [f for f in mpbuild.flags() if f not in ("-shared", "-fPIC")]
    res = subprocess.run([mpbuild.hipcc(), *flags, f"-ffp-contract={contract}", "-I", mpbuild.CSRC,
                          "--cuda-device-only", "-S", str(src), "-o", str(out)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    asm = out.read_text()
    assert len(re.findall(r"\bv_(?:fma|fmac|fmaak|fmamk)_f32", asm)) == 1
    assert len(re.findall(r"\bv_mul_f32", asm)) == 1 and not re.findall(r"\bv_add_f32", asm)


@pytest.mark.parametrize("fn,defaults,rows", [
    (mp.mpgemm_quantize_rows, QUANT, dict(T=0, R=0)), (mp.mpgemm_gather_rows, GATHER, dict(R=0)),
    (mp.mpgemm_combine_rows, COMBINE, dict(T=0)), (mp.mpgemm_combine_rows_backward, BACK, dict(T=0))])
def test_widest_row(fn, defaults, rows):
    """The one limit on H that the header states holds for every row function."""
    text = open(os.path.join(ROOT, "include", "mpgemm_ops.h")).read()
    assert "row has at\n * most 2^28 values" in text and not re.search(r"\bH\b[^.;]*below 2\^31", text)
    wide = {n: 1 << 29 for n in defaults if n.startswith("ld")}
    assert call(fn, defaults, H=1 << 28, **rows, **wide) == 0
    assert call(fn, defaults, H=(1 << 28) + 1, **rows, **wide) == mp.MPGEMM_EDIM
