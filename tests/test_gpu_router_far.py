"""GPU: the router's calls on rows that lie past 2^32 elements of their tensors
give the bits of the same calls on contiguous rows."""
import pytest
import torch

import dense_mixed_precision_amd as mp
from tests.gpu_util import device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k,dtype", [(40, 4, torch.bfloat16), (300, 20, torch.float16)])
def test_rows_past_32_bits(E, k, dtype):
    dev, T, ld = device(), 2500, 1 << 21
    assert (T - 1) * ld > 1 << 32
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(E)).to(dtype).to(dev)
    x[7] = -torch.inf
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(k)).to(dev)

    def rows():
        return torch.empty((T - 1) * ld + E, dtype=dtype, device=dev).as_strided((T, E), (ld, 1))

    def step(logits, dlogits, normalize):
        ids, w = torch.empty(T, k, dtype=torch.int32, device=dev), torch.empty(T, k, device=dev)
        loss, probs = torch.empty(1, device=dev), torch.empty(E, device=dev)
        counts = torch.empty(E + 1, dtype=torch.int32, device=dev)
        mp.select_experts(logits, ids, w, normalize=normalize)
        mp.balance_loss(logits, ids, loss, counts, probs=probs)
        mp.router_backward(logits, ids, dlogits, dweights=dw, normalize=normalize, counts=counts)
        torch.cuda.synchronize()
        return ids, w, loss, counts, probs, dlogits.contiguous()

    far, dfar = rows(), rows()
    far.copy_(x)
    for normalize in (True, False):
        near = step(x, torch.empty_like(x), normalize)
        assert int(near[3][E]) == T - 1 and bool((near[5] != 0).any())
        assert all(torch.equal(a, b) for a, b in zip(step(far, dfar, normalize), near))
