"""GPU: gradients of pairs that have no weight.  What stands in dweights at a
pair without an expert, at one whose expert's logit is -inf, or in a row that is
-inf throughout (garbage, infinities, NaN) changes nothing: the gradient is the
one with zeros there, to the bit."""
import math

import pytest
import torch

import dense_mixed_precision_amd as mp
from tests.gpu_util import device

pytestmark = pytest.mark.gpu
INF = math.inf


def masked_case(T, E, k, dtype, seed):
    """(logits, ids, truth values: the pair has a weight): experts masked at
    random, row 1 whole; ids of masked experts, of none, and outside among the
    others, the same expert twice."""
    g = torch.Generator().manual_seed(seed)
    x = 2.0 * torch.randn(T, E, generator=g)
    x[torch.rand(T, E, generator=g) < 0.3] = -INF
    x[1] = -INF
    ids = torch.randint(0, E, (T, k), generator=g)
    ids[torch.rand(T, k, generator=g) < 0.1] = -1
    ids[torch.rand(T, k, generator=g) < 0.1] = E
    there = (ids >= 0) & (ids < E)
    there &= x.gather(1, ids.clamp(0, E - 1)) > -INF
    assert bool(there.any()) and not bool(there.all())
    return x.to(dtype).to(device()), ids.to(device()), there.to(device())


@pytest.mark.parametrize("garbage", [math.nan, INF, -INF, 3.0e38])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("balance", [True, False])
@pytest.mark.parametrize("T,E,k,dtype", [
    (40, 13, 4, torch.float32), (37, 100, 8, torch.bfloat16), (21, 256, 20, torch.float16), (19, 300, 6, torch.float32),
    (9, 1024, 64, torch.bfloat16)])
def test_dweights_without_a_weight_are_not_looked_at(garbage, normalize, balance, T, E, k, dtype):
    x, ids, there = masked_case(T, E, k, dtype, T + E)
    counts = None
    if balance:
        counts = torch.empty(E + 1, dtype=torch.int32, device=device())
        mp.balance_loss(x, ids, torch.empty(1, device=device()), counts)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(k)).to(device())
    got = torch.empty(T, E, device=device())
    want = torch.empty_like(got)
    mp.router_backward(x, ids, want, dweights=torch.where(there, dw, 0.0), normalize=normalize, counts=counts)
    mp.router_backward(x, ids, got, dweights=torch.where(there, dw, garbage), normalize=normalize, counts=counts)
    torch.cuda.synchronize()
    assert torch.isfinite(want).all() and bool((want != 0).any())
    assert torch.equal(got, want)
    assert not bool(want[x == -INF].any())


@pytest.mark.parametrize("normalize", [True, False])
def test_dweights_with_a_weight_reach_their_token_only(normalize):
    """A NaN at a pair that has a weight makes its own token's gradient NaN."""
    x, ids, there = masked_case(40, 60, 3, torch.float32, 3)
    t = int(there[2:, 1].nonzero()[0]) + 2
    dw = torch.where(there, 1.5, 0.0)
    clean, got = torch.empty(40, 60, device=device()), torch.empty(40, 60, device=device())
    mp.router_backward(x, ids, clean, dweights=dw, normalize=normalize)
    dw[t, 1] = math.nan
    mp.router_backward(x, ids, got, dweights=dw, normalize=normalize)
    torch.cuda.synchronize()
    chosen = ids[t][there[t]]
    assert torch.isnan(got[t, chosen]).all()
    rest = torch.arange(40, device=device()) != t
    assert torch.equal(got[rest], clean[rest])
