"""GPU: the largest BF16 tokens that no group's sum of 4-bit products can make
overflow."""
import pytest
import torch

import dense_mixed_precision_amd as mp
from tests.gpu_util import device
from tests.w4_util import pack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("M,N", [(3, 20), (16, 4700), (30, 8100), (61, 9001), (70, 12500), (63, 41001), (130, 24601)])
def test_tokens_below_2_to_122_do_not_overflow(M, N, group):
    """All of a group's products at their largest and of one sign, with a scale
    that brings the result back: exact, since each sum is a whole number below
    2^20 of a power of two."""
    dev, K = device(), 256
    top = 255.0 * 2.0 ** 114              # the largest BF16 number below 2^122
    a = torch.full((M, K), top, dtype=torch.bfloat16, device=dev)
    a[M // 2] = -top
    q = pack(torch.full((1, K), -8, dtype=torch.int64)).expand(N, -1).contiguous().to(dev)
    scale = torch.full((N, -(-K // group)), 2.0 ** -60, dtype=torch.bfloat16, device=dev)
    out = torch.empty(M, N, device=dev)
    mp.gemm_w4(a, q, scale, out, group=group)
    want = torch.full((M, 1), -8.0 * K * 255.0 * 2.0 ** 54, device=dev)
    want[M // 2] *= -1
    torch.cuda.synchronize()
    assert float(a[0, 0]) == top and torch.equal(out, want.expand(M, N))
