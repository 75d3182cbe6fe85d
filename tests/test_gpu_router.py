"""GPU: the router -- selection, balance loss, and their gradient -- against
the definitions in 64 bits.

Bounds (u = 2^-24).  The difference d <= 0 of two FP32 logits is rounded, which
changes exp(d) by u*|d| of itself: |d| < 88 where exp(d) is a normal number
(above 2^-126 = exp(-87.3)), and |d|*exp(d) < 0.37 of the largest term in a sum.
The power of two is off by 2u, the products and corrections around it by 6u.  A
sum of n terms adds n*u and its terms' own 8u + 0.37n*u; the quotient u.  So a
probability is off by (88 + 8 + 8 + 1.37*E + 1)*u < (106 + 2*E)*u = rel(E) of
itself, plus 2^-126 where it is taken for 0."""
import math

import pytest
import torch

import dense_mixed_precision_amd as mp
from tests.gpu_util import device
from tests.ops_util import HALF_STEP, TINY, U32, Buffer, assert_within

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = [F16, BF16, F32]
INF = math.inf


def rel(E):
    return (106 + 2 * E) * U32 * 1.01


def softmax(x):
    """In 64 bits on the CPU; zeros for a row of -inf, NaN with a NaN or +inf."""
    x = x.double()
    top = x.amax(1, keepdim=True) if x.shape[1] else x.new_full((x.shape[0], 1), -INF)
    e = torch.where(top > -INF, torch.exp(x - torch.where(top > -INF, top, 0.0)), 0.0)
    p = e / torch.where(top > -INF, e.sum(1, keepdim=True), 1.0)
    bad = torch.isnan(x).any(1, keepdim=True) | (x == INF).any(1, keepdim=True)
    return torch.where(bad, math.nan, p)


def chosen(x, k):
    """ids by definition, one token at a time."""
    out = []
    for row in x.double().tolist():
        order = sorted((e for e, v in enumerate(row) if v != -INF),
                       key=lambda e: (-INF if math.isnan(row[e]) else 0, 0 if math.isnan(row[e]) else -row[e], e))
        out.append((order + [-1] * k)[:k])
    return torch.tensor(out, dtype=torch.int64).reshape(len(out), k)


def weights_of(x, ids, normalize):
    """(weights, their relative bound) of given pairs."""
    E = x.shape[1]
    there = (ids >= 0) & (ids < E)
    at = ids.clamp(0, E - 1)
    if not normalize:
        return torch.where(there, softmax(x).gather(1, at), 0.0), rel(E)
    return softmax(torch.where(there, x.double().gather(1, at), -INF)), rel(ids.shape[1])


def logits(T, E, dtype, seed, masked=0.1, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn(T, E, generator=g)
    x[torch.rand(T, E, generator=g) < masked] = -INF
    if T > 2:
        x[1] = -INF
    return x.to(dtype)


def check_weights(got, x, ids, normalize, what):
    want, r = weights_of(x, ids, normalize)
    nan = torch.isnan(want)
    there = ids >= 0
    want = torch.where(there, want, 0.0)
    got = got.cpu()
    assert torch.equal(torch.isnan(got), nan & there), what
    clean = torch.where(nan, 0.0, want)
    assert_within(torch.nan_to_num(got), clean, r * clean + 2.0 ** -126, what)


def check_select(x, k, normalize, gap=0, shift=0):
    T, E = x.shape
    X = Buffer(T, E, x.dtype, x, gap, shift)
    ids = Buffer(1, T * k, torch.int32, shift=shift)
    w = Buffer(1, T * k, F32, shift=shift)
    mp.select_experts(X.view, ids.view.reshape(T, k), w.view.reshape(T, k), normalize=normalize)
    torch.cuda.synchronize()
    want = chosen(x, k)
    assert torch.equal(ids.view.reshape(T, k).cpu().long(), want)
    check_weights(w.view.reshape(T, k), x, want, normalize, f"{T}x{E} top {k}")
    assert ids.outside_untouched() and w.outside_untouched()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,gap,shift", [
    (1, 1, 1, 0, 0), (3, 2, 2, 1, 1), (5, 13, 2, 0, 0), (17, 16, 16, 0, 0), (33, 17, 3, 3, 1), (16, 32, 8, 0, 0),
    (64, 60, 4, 0, 0), (7, 64, 17, 1, 0), (50, 100, 10, 0, 1), (200, 128, 8, 0, 0), (9, 200, 16, 5, 1), (31, 256, 5, 0, 0),
    (8, 256, 64, 0, 0), (21, 300, 9, 0, 0), (6, 512, 64, 2, 1), (13, 1000, 33, 1, 1), (5, 1024, 8, 0, 0), (0, 8, 2, 0, 0)])
def test_select(dtype, normalize, T, E, k, gap, shift):
    check_select(logits(T, E, dtype, T * 131 + E), k, normalize, gap, shift)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E", [5, 40, 130, 700])
@pytest.mark.parametrize("normalize", [True, False])
def test_select_ties_and_extremes(dtype, E, normalize):
    info = torch.finfo(dtype)
    g = torch.Generator().manual_seed(E)
    x = torch.randint(-2, 3, (14, E), generator=g).double()   # many equal ones
    x[1] = 0.0
    x[1, ::2] = -0.0
    x[2] = info.min                                           # the lowest number is a number
    x[3] = -INF
    x[4] = -INF
    x[4, E // 2] = info.min
    x[5], x[5, 0] = info.min, info.max
    x[6, E - 1] = math.nan
    x[7, E - 2], x[7, 1] = INF, INF
    x[8, 2], x[8, 3] = math.nan, INF
    x[9] = -INF
    x[9, 1:3] = torch.tensor([-1.0, -1.0])
    x[10] = info.tiny * info.eps * torch.arange(E)            # below the normal numbers
    x[11] = -100.0 * torch.arange(E)
    x[12] = 60.0 * torch.randn(E, generator=g)
    check_select(x.to(dtype), min(E, 4), normalize)


def definition_balance(x, ids, coefficient):
    E = x.shape[1]
    p = softmax(x)
    counts = torch.tensor([int((ids == e).sum()) for e in range(E)], dtype=torch.int64)
    tokens = int((x.double() != -INF).any(1).sum()) if x.shape[0] else 0
    probs = p.sum(0)
    pairs = int(counts.sum())
    share = counts.double() * (coefficient * E / (pairs * tokens)) if pairs and tokens else torch.zeros(E).double()
    return p, counts, tokens, probs, share


def some_ids(T, E, k, seed, dtype=torch.int32):
    """Pairs with absent ones, ids outside, and the same expert twice."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g)
    ids[torch.rand(T, k, generator=g) < 0.1] = -1
    ids[torch.rand(T, k, generator=g) < 0.03] = E
    return ids.to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k,gap,shift,id_type", [
    (1, 1, 1, 0, 0, torch.int32), (5, 3, 2, 1, 1, torch.int64), (64, 13, 2, 0, 0, torch.int32),
    (65, 16, 4, 0, 0, torch.int32), (1000, 60, 1, 0, 1, torch.int64), (300, 100, 8, 3, 0, torch.int32),
    (2000, 128, 8, 0, 0, torch.int32), (129, 256, 20, 0, 0, torch.int64), (700, 257, 3, 1, 1, torch.int32),
    (333, 1024, 6, 0, 0, torch.int32), (40000, 33, 2, 0, 0, torch.int32), (0, 8, 2, 0, 0, torch.int32),
    (9, 8, 0, 0, 0, torch.int32)])
def test_balance(dtype, T, E, k, gap, shift, id_type):
    x = logits(T, E, dtype, T + E)
    ids = some_ids(T, E, k, T * 3 + E, id_type)
    X = Buffer(T, E, dtype, x, gap, shift)
    loss, counts, probs = Buffer(1, 1, F32), Buffer(1, E + 1, torch.int32), Buffer(1, E, F32)
    mp.balance_loss(X.view, ids.to(device()), loss.view.reshape(1), counts.view.reshape(-1), probs=probs.view.reshape(-1),
                    coefficient=0.25)
    torch.cuda.synchronize()
    p, want, tokens, psum, share = definition_balance(x, ids.long(), 0.25)
    assert counts.view.reshape(-1).cpu().tolist() == want.tolist() + [tokens]
    # a sum of T probabilities: T roundings at most, whatever their order
    err = (rel(E) + T * U32) * 1.01 * psum + T * 2.0 ** -126
    assert_within(probs.view.reshape(-1), psum, err, "probs")
    # the products of counts (rounded) and sums, their sum, and three more roundings
    total = (share * psum).sum().reshape(1)
    assert_within(loss.view.reshape(-1), total, (share * err).sum() + (E + 10) * U32 * 1.01 * total, "loss")
    for b in (loss, counts, probs):
        assert b.outside_untouched()


def definition_backward(x, ids, dw, normalize, share, dloss):
    """(gradient, sum of the magnitudes that make it) in 64 bits."""
    E = x.shape[1]
    p = softmax(x)
    u = torch.zeros_like(p)
    d, dmag = torch.zeros_like(p), torch.zeros_like(p)
    umag = torch.zeros_like(p)
    if share is not None:
        u += dloss * share
        umag += abs(dloss) * share
    if dw is not None:
        there = (ids >= 0) & (ids < E)
        at, v = ids.clamp(0, E - 1), torch.where(there, dw.double(), 0.0)
        if normalize:
            w = weights_of(x, ids, True)[0]
            mean, mmag = (w * v).sum(1, keepdim=True), (w * v.abs()).sum(1, keepdim=True)
            d.scatter_add_(1, at, w * (v - mean))
            dmag.scatter_add_(1, at, w * (v.abs() + mmag))
        else:
            u.scatter_add_(1, at, v)
            umag.scatter_add_(1, at, v.abs())
    out = p * (u - (p * u).sum(1, keepdim=True)) + d
    return out, p * (umag + (p * umag).sum(1, keepdim=True)) + dmag


@pytest.mark.parametrize("dtype,dtype_d", [(F32, F32), (BF16, BF16), (F16, F32), (F32, F16), (BF16, F32)])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("parts", ["weights", "loss", "both"])
@pytest.mark.parametrize("T,E,k,gap,shift,id_type", [
    (1, 1, 1, 0, 0, torch.int32), (5, 3, 2, 1, 1, torch.int64), (33, 16, 16, 0, 0, torch.int32),
    (40, 60, 5, 0, 1, torch.int64), (100, 128, 8, 0, 0, torch.int32), (70, 200, 3, 3, 0, torch.int32),
    (9, 256, 17, 0, 0, torch.int64), (21, 300, 9, 1, 1, torch.int32), (6, 1024, 64, 0, 0, torch.int32),
    (0, 8, 2, 0, 0, torch.int32), (33000, 7, 2, 0, 0, torch.int32)])
def test_backward(dtype, dtype_d, normalize, parts, T, E, k, gap, shift, id_type):
    x = logits(T, E, dtype, T + 2 * E)
    ids = some_ids(T, E, k, T * 5 + E, id_type)
    g = torch.Generator().manual_seed(T + k)
    dw = torch.randn(T, k, generator=g) if parts != "loss" else None
    share, counts, dloss = None, None, None
    if parts != "weights":
        _, c, tokens, _, share = definition_balance(x, ids.long(), 0.5)
        counts = torch.tensor(c.tolist() + [tokens], dtype=torch.int32, device=device())
        dloss = torch.tensor([-1.5], device=device())
    X, D = Buffer(T, E, dtype, x, gap, shift), Buffer(T, E, dtype_d, gap=gap, shift=shift)
    mp.router_backward(X.view, None if dw is None else ids.to(device()), D.view,
                       dweights=None if dw is None else dw.to(device()), normalize=normalize, counts=counts, dloss=dloss,
                       coefficient=0.5)
    torch.cuda.synchronize()
    want, mag = definition_backward(x, ids.long(), dw, normalize, share, -1.5)
    # every factor is a probability or weight, a gradient (k added up, the loss's
    # with 5 roundings and a sum of E counts) or a sum of their products
    err = (2 * rel(E) + 2 * rel(k) + (3 * E + 2 * k + 20) * U32) * 1.01 * mag + 2.0 ** -120
    assert_within(D.view, want, err + HALF_STEP[dtype_d] * (want.abs() + err) + TINY[dtype_d], f"{T}x{E} top {k} {parts}")
    assert D.outside_untouched()
