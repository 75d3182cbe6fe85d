"""Host-side tests of the operator library at its edges (no GPU): slots a
token beyond what the kernels' counters hold."""
import pytest

import dense_mixed_precision_amd as mp
from tests.test_ops_host import COMBINE, call

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
