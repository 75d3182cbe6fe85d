"""GPU: the arithmetic behind the exact sum of the 8-bit product, bit by bit.
With s the sum rounded to FP32 and v = fl(s * scale_a), an FP32 result is
fl(v * scale_b) without a bias and fl(v * scale_b + bias), rounded once, with
one."""
import pytest
import torch

import dense_mixed_precision_amd as mp
from tests.gpu_util import device
from tests.ops_util import offsets_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,sizes", [(3, 20, 64, None), (16, 16400, 520, None), (300, 1000, 400, None),
                                         (500, 1000, 333, None), (600, 2000, 77, None), (1500, 1400, 200, None),
                                         (2040, 4000, 600, None), (2600, 4100, 141, None),
                                         (70, 72, 144, [3, 0, 67]), (2500, 1100, 200, [1, 700, 0, 1299, 490])])
def test_scales_and_bias_round_as_stated(M, N, K, sizes):
    """The bias is minus the rounded product, the same for every row: the sum
    is what rounding the product lost, at most 24 bits of the 48 that 64-bit
    numbers hold, so the expected value is exact.  Two roundings give 0."""
    g = torch.Generator().manual_seed(M + N + K)
    a = torch.randint(-127, 128, (1, K), generator=g, dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8)
    sa, sb = torch.rand(1, generator=g) + 0.5, torch.rand(N, generator=g) + 0.5
    v = (a.long() @ w.long().t())[0].float() * sa
    plain = v * sb
    lost = v.double() * sb.double() - plain.double()
    assert (lost != 0).float().mean() > 0.5
    dev = device()
    A, SA = a.expand(M, K).contiguous().to(dev), sa.expand(M).contiguous().to(dev)
    W, SB, B = w.to(dev).t(), sb.to(dev), (-plain).to(dev)
    offsets = None
    if sizes is not None:
        G = len(sizes)
        W, SB, B = W.expand(G, K, N), SB.expand(G, N).contiguous(), B.expand(G, N).contiguous()
        offsets = offsets_of(sizes)
    out, fused = torch.empty(M, N, device=dev), torch.empty(M, N, device=dev)
    mp.gemm_i8(A, W, out, SA, SB, offsets=offsets)
    mp.gemm_i8(A, W, fused, SA, SB, bias=B, offsets=offsets)
    torch.cuda.synchronize()
    R = M if sizes is None else sum(sizes)  # rows of no group keep what they hold
    assert torch.equal(out.cpu()[:R], plain.expand(R, N))
    assert torch.equal(fused.cpu().double()[:R], lost.expand(R, N))
