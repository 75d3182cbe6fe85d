"""GPU: the gradient by the tokens of products with 4-bit weights, dX = dY W, by
way of dequantize_w4 and the 16-bit products, one matrix and one per expert."""
import pytest
import torch

import dense_mixed_precision_amd as mp
from tests.gpu_util import device
from tests.ops_util import HALF_STEP, U32, assert_within, offsets_of
from tests.w4_util import random_weights, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("sizes,N,K,group", [([7], 96, 200, 32), ([0, 5, 33, 1], 70, 129, 64), ([64, 0, 300], 256, 512, 128)])
def test_tokens_gradient(dtype, sizes, N, K, group):
    """Each weight, code * scale (exact in FP32), is rounded to the type: half a
    step of it.  The product's sum of N FP32 terms is off by a step (2u) each."""
    dev, G, R = device(), len(sizes), sum(sizes)
    g = torch.Generator().manual_seed(R + N)
    _, packed, scale = random_weights(g, N, K, group, dtype, G)
    dy = torch.randn(R, N, generator=g).to(dtype)
    q, s, w = packed.to(dev), scale.to(dev), torch.empty(G, N, K, dtype=dtype, device=dev)
    for e in range(G):
        mp.dequantize_w4(q[e], s[e], w[e], group=group)
    dx = torch.empty(R, K, device=dev)
    if G == 1:
        mp.gemm(dy.to(dev), w[0], dx)
    else:
        mp.gemm_grouped(dy.to(dev), w, dx, offsets_of(sizes))
    torch.cuda.synchronize()
    at = 0
    for e, n in enumerate(sizes):
        here, v = slice(at, at + n), values(packed[e], scale[e], K, group)
        want, mag = dy[here].double() @ v, dy[here].double().abs() @ v.abs()
        assert_within(dx[here], want, (HALF_STEP[dtype] + 2 * N * U32) * 1.01 * mag, f"expert {e}")
        at += n
