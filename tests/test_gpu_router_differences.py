"""GPU: the router's gradient against differences, at every logit: the rows'
logits lie further apart than the steps, so no step changes the selection."""
import pytest
import torch

import dense_mixed_precision_amd as mp
from tests.gpu_util import device
from tests.ops_util import U32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(6, 9, 3), (2, 40, 5), (2, 20, 18)])
def test_every_logit(normalize, T, E, k):
    """Central differences of the framework's own weights and loss with step h.
    What a row adds to either is f = <s, softmax> (s the weights' gradients, or
    the loss's pull on each expert), whose third derivative by a logit is
    p (1 - 6p + 6p^2) (s_e - f), at most 2 max|s|: the difference leaves h^2 / 6 of
    that.  A probability is off by (4 + 8 + 8 + 1.37 E + 1)u < 76u of itself, for
    logits less than 4 apart (see test_gpu_router), the loss by (E + 16)u more:
    160u of the value, over h."""
    dev, h = device(), 2.0 ** -5
    g = torch.Generator().manual_seed(T + E)
    # rows of the same values in different orders, 3/32 apart: h adds exactly
    order = torch.stack([torch.randperm(E, generator=g) for _ in range(T)])
    x = ((order - E // 2) * 0.09375).to(dev)
    dw = torch.randn(T, k, generator=g).to(dev)
    ids, w = torch.empty(T, k, dtype=torch.int32, device=dev), torch.empty(T, k, device=dev)
    loss, counts = torch.empty(1, device=dev), torch.empty(E + 1, dtype=torch.int32, device=dev)
    mp.select_experts(x, ids, w, normalize=normalize)
    mp.balance_loss(x, ids, loss, counts, coefficient=2.0)
    dx, dloss = torch.empty_like(x), torch.tensor([3.0], device=dev)
    mp.router_backward(x, ids, dx, dweights=dw, normalize=normalize, counts=counts, dloss=dloss, coefficient=2.0)
    assert torch.equal(ids.cpu().long(), order.argsort(1, descending=True)[:, :k])

    def values(y):
        ids2, w2, l2, c2 = torch.empty_like(ids), torch.empty_like(w), torch.empty_like(loss), torch.empty_like(counts)
        mp.select_experts(y, ids2, w2, normalize=normalize)
        mp.balance_loss(y, ids, l2, c2, coefficient=2.0)
        assert torch.equal(ids2, ids) and torch.equal(c2, counts)
        return (w2.double() * dw.double()).sum(1), 3.0 * float(l2)

    third, rounding = h * h / 3, 160 * U32 / h
    pull = 3.0 * 2.0 * E * float(counts[:E].max()) / (T * k * T)
    compared = 0
    for t in range(T):
        bound = ((third + rounding) * float(dw[t].abs().max()) + third * pull + rounding * 3.0 * 1.1 * float(loss))
        # (far below the gradient: one of zeros would not pass)
        assert float(dx[t].abs().max()) > 5 * bound
        for e in range(E):
            up, down = x.clone(), x.clone()
            up[t, e] += h
            down[t, e] -= h
            (wu, lu), (wd, ld) = values(up), values(down)
            diff = (float(wu[t] - wd[t]) + lu - ld) / (2 * h)
            assert abs(diff - float(dx[t, e])) <= bound, (t, e)
            compared += 1
    assert compared == T * E
