"""GPU: pairs sorted by expert, rows into that order and back with their
gradients, and the experts' 16-bit products with theirs, against the
definitions in 64 bits.

Bounds (u = 2^-24, h the output type's half step): a weighted sum of k rows is
k fused steps in FP32, k*u of the sum of magnitudes, and h of the result.  A
dot product over H values takes at most ceil(H/64) + 16 FP32 additions in a
chain (64 lanes: 8 per whole 512 values, one more and 6 across lanes; 16 lanes
up to H = 256: 16, one more where H is no multiple of 8, and 4 across).  A grouped product is an FP32 running sum of K products: (K + 2)*u of
the sum of magnitudes covers any order and the epilogue's alpha and beta."""
import pytest
import torch

import dense_mixed_precision_amd as mp
from tests.gpu_util import device
from tests.ops_util import HALF_STEP, TINY, U32, Buffer, assert_within, offsets_of, order_by_expert

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16, torch.float32]


def make_ids(T, k, E, seed, dtype=torch.int32, drop=0.0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g)
    if drop:
        ids = torch.where(torch.rand(T, k, generator=g) < drop, torch.randint(-3, 0, (T, k), generator=g), ids)
    return ids.to(dtype)


def check_route(ids, E):
    order, position, offsets = mp.route(ids.to(device()), E)
    torch.cuda.synchronize()
    want = order_by_expert(ids, E)
    assert offsets.tolist() == want[2]
    assert order.tolist() == want[0]
    assert position.shape == ids.shape and position.reshape(-1).tolist() == want[1]


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 8, 8), (3, 2, 1000), (64, 4, 64), (255, 3, 7),
                                   (1024, 4, 16), (1025, 4, 16), (4097, 1, 128), (5000, 8, 128), (40000, 8, 1024),
                                   (9001, 2, 1), (70001, 8, 5)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_route_sizes(T, k, E, dtype):
    check_route(make_ids(T, k, E, T + k + E, dtype), E)


@pytest.mark.parametrize("T", [50, 9000])
def test_route_dropped_and_outside(T):
    check_route(make_ids(T, 4, 9, T, drop=0.4), 9)
    check_route(torch.full((T, 4), -1, dtype=torch.int32), 9)       # no pair has an expert
    check_route(torch.full((T, 4), 8, dtype=torch.int64), 9)        # all the last one
    ids = make_ids(T, 4, 20, T + 1, torch.int64)                    # half beyond the experts
    ids[0, 0], ids[1, 1], ids[2, 2] = 1 << 40, -(1 << 40), 1 << 32  # whose low 32 bits are in range
    check_route(ids, 9)


def test_route_out_workspace_stream():
    ids = make_ids(3000, 4, 33, 2).to(device())
    out = (torch.empty(12000, dtype=torch.int32, device=device()),
           torch.empty(3000, 4, dtype=torch.int32, device=device()),
           torch.empty(34, dtype=torch.int32, device=device()))
    need = mp.mpgemm_route_workspace(12000, 33)
    ws = torch.empty(need // 4, dtype=torch.int32, device=device())
    got = mp.route(ids, 33, out=out, workspace=ws)
    assert got[0] is out[0] and got[2] is out[2]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = mp.route(ids, 33, stream=side)
    torch.cuda.synchronize()
    want = order_by_expert(ids.cpu(), 33)
    for g in (got, other):
        assert g[0].tolist() == want[0] and g[1].reshape(-1).tolist() == want[1] and g[2].tolist() == want[2]
    with pytest.raises(mp.MpgemmError):
        mp.route(ids, 33, workspace=ws[:10])


def test_route_refuses_wrong_out():
    ids = make_ids(3, 2, 4, 1).to(device())
    good = [torch.empty(n, dtype=torch.int32, device=device()) for n in ((6,), (3, 2), (5,))]
    for i, wrong, error in ((0, None, TypeError), (1, [0] * 6, TypeError), (2, good[2].float(), TypeError),
                            (1, good[0], ValueError), (2, good[2][:4], ValueError), (0, good[0].cpu(), ValueError)):
        out = list(good)
        out[i] = wrong
        with pytest.raises(error):
            mp.route(ids, 4, out=out)
    with pytest.raises(ValueError):
        mp.route(ids, 4, out=good[:2])
    with pytest.raises(ValueError):
        mp.route(ids, 4, workspace=torch.zeros(64, dtype=torch.int32))


def test_route_graph():
    for T in (100, 3000):
        ids = make_ids(T, 4, 33, 2).to(device())
        mp.route(ids, 33)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = mp.route(ids, 33)
        for r in range(3):
            ids.copy_(make_ids(T, 4, 33, 50 + r, drop=0.2))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            want = order_by_expert(ids.cpu(), 33)
            assert got[0].tolist() == want[0] and got[1].reshape(-1).tolist() == want[1] and got[2].tolist() == want[2]


# ---- rows -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,H,gap,shift", [(1, 1, 1, 1, 0, 0), (5, 2, 3, 7, 1, 1), (33, 8, 64, 256, 0, 0),
                                               (20, 3, 4, 1025, 3, 1), (9, 2, 5, 2048, 0, 0), (4, 2, 3, 0, 0, 0),
                                               (40, 2, 5, 128, 0, 0), (21, 2, 5, 129, 1, 0)])
def test_gather_rows(dtype, T, k, E, H, gap, shift):
    ids = make_ids(T, k, E, T + H, drop=0.2)
    order, _, offsets = mp.route(ids.to(device()), E)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(dtype)
    X, Y = Buffer(T, H, dtype, x, gap, shift), Buffer(T * k, H, dtype, gap=gap, shift=shift)
    mp.gather_rows(X.view, order, Y.view, top_k=k)
    torch.cuda.synchronize()
    want = Y.before.clone()
    wv = torch.as_strided(want, Y.view.shape, Y.view.stride(), Y.view.storage_offset())
    for p, i in enumerate(order.tolist()):
        if i >= 0:
            wv[p] = X.view[i // k]
    assert torch.equal(Y.flat, want)


@pytest.mark.parametrize("dtype,T,k,H,gap,shift", [(torch.bfloat16, 6000, 3, 2051, 1, 1), (torch.float32, 4100, 2, 2304, 0, 0),
                                                   (torch.float16, 700, 9, 6000, 8, 0)])
def test_gather_many_rows(dtype, T, k, H, gap, shift):
    """Rows enough for the way by tokens, equal to the way by rows, also where
    the order is no permutation: pairs absent, twice, outside."""
    g = torch.Generator().manual_seed(H)
    order, _, _ = mp.route(make_ids(T, k, 37, H, drop=0.1).to(device()), 37)
    R = T * k
    assert mp.mpgemm_rows_workspace(mp.MPGEMM_T_F32 if dtype == torch.float32 else 0, T, H, R, k) > 0
    x = torch.randn(T, H, generator=g).to(dtype)
    X, Y = Buffer(T, H, dtype, x, gap, shift), Buffer(R, H, dtype, gap=gap, shift=shift)
    want = Y.before.clone()
    wv = torch.as_strided(want, Y.view.shape, Y.view.stride(), Y.view.storage_offset())
    for odd in (False, True):
        if odd:
            order[5], order[R // 2], order[R // 3] = order[0], order[0], order[1]
            order[7], order[8], order[9] = R, -2, (1 << 31) - 1
            Y.flat.copy_(Y.before)
            want.copy_(Y.before)
        mp.gather_rows(X.view, order, Y.view, top_k=k)
        torch.cuda.synchronize()
        there = (order >= 0) & (order < R)
        wv[there] = X.view[(order[there] // k).long()]
        assert torch.equal(Y.flat, want)


def test_gather_rows_wrong_indices():
    X = Buffer(4, 32, torch.float32, torch.randn(4, 32))
    Y = Buffer(6, 32, torch.float32)
    order = torch.tensor([8, 7, -1, -(1 << 31), (1 << 31) - 1, 7], dtype=torch.int32, device=device())
    mp.gather_rows(X.view, order, Y.view, top_k=2)
    torch.cuda.synchronize()
    want = torch.full((6, 32), -12345.5, device=device())
    want[1] = want[5] = X.view[3]
    assert torch.equal(Y.view, want) and Y.outside_untouched()


def combine_exact(y, position, w, T, H):
    exact, size = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for s in range(position.shape[1]):
            p = int(position[t, s])
            if p >= 0:
                v = float(w[t, s]) * y[p].double()
                exact[t] += v
                size[t] += v.abs()
    return exact, size


@pytest.mark.parametrize("yt", DTYPES)
@pytest.mark.parametrize("ot", DTYPES)
@pytest.mark.parametrize("T,k,E,H,gap,shift", [(1, 1, 1, 1, 0, 0), (6, 2, 3, 7, 1, 1), (17, 8, 64, 256, 0, 0),
                                               (33, 5, 4, 64, 0, 0), (18, 3, 4, 129, 1, 0), (7, 9, 4, 513, 0, 1),
                                               (5, 3, 4, 2051, 2, 1)])
def test_combine_rows(yt, ot, T, k, E, H, gap, shift):
    g = torch.Generator().manual_seed(T + H)
    ids = make_ids(T, k, E, T + H, drop=0.25)
    _, position, _ = mp.route(ids.to(device()), E)
    y, w = torch.randn(T * k, H, generator=g).to(yt), torch.rand(T, k, generator=g) - 0.3
    Y, O = Buffer(T * k, H, yt, y, gap, shift), Buffer(T, H, ot, gap=gap, shift=shift)
    for weights in (w, None):
        mp.combine_rows(Y.view, position, O.view, weights=None if weights is None else w.to(device()))
        torch.cuda.synchronize()
        exact, size = combine_exact(y, position, torch.ones_like(w) if weights is None else w, T, H)
        bound = k * U32 * 1.01 * size
        assert_within(O.view, exact, bound + HALF_STEP[ot] * (exact.abs() + bound) + TINY[ot], "combine")
        assert O.outside_untouched() and torch.equal(Y.flat, Y.before)


def test_combine_no_slots_no_rows_wrong_positions():
    O = Buffer(3, 40, torch.float32)
    Y = Buffer(5, 40, torch.float32, torch.randn(5, 40))
    none = torch.empty(3, 0, dtype=torch.int32, device=device())
    mp.combine_rows(Y.view, none, O.view)
    torch.cuda.synchronize()
    assert (O.view == 0).all() and O.outside_untouched()
    at = torch.tensor([[0, 5], [-1, -9], [(1 << 31) - 1, 4]], dtype=torch.int32, device=device())
    mp.combine_rows(Y.view, at, O.view)
    torch.cuda.synchronize()
    assert torch.equal(O.view[0], Y.view[0]) and (O.view[1] == 0).all() and torch.equal(O.view[2], Y.view[4])
    mp.combine_rows(Y.view[:0], at, O.view)
    torch.cuda.synchronize()
    assert (O.view == 0).all()


@pytest.mark.parametrize("dt,yt,gt", [(torch.float32, torch.float32, torch.float32),
                                      (torch.bfloat16, torch.float32, torch.bfloat16),
                                      (torch.float16, torch.float16, torch.float16),
                                      (torch.bfloat16, torch.bfloat16, torch.float32),
                                      (torch.float32, torch.float16, torch.bfloat16)])
@pytest.mark.parametrize("T,k,E,H,gap,shift", [(1, 1, 1, 1, 0, 0), (6, 2, 3, 7, 1, 1), (17, 8, 64, 256, 0, 0),
                                               (9, 5, 4, 119, 0, 0), (7, 3, 4, 264, 0, 0), (5, 3, 4, 2051, 2, 1)])
def test_combine_rows_backward(dt, yt, gt, T, k, E, H, gap, shift):
    g = torch.Generator().manual_seed(T + H)
    ids = make_ids(T, k, E, T + H, drop=0.25)
    order, position, offsets = mp.route(ids.to(device()), E)
    d, y = torch.randn(T, H, generator=g).to(dt), torch.randn(T * k, H, generator=g).to(yt)
    w = torch.rand(T, k, generator=g) - 0.3
    D, Y, G = Buffer(T, H, dt, d, gap, shift), Buffer(T * k, H, yt, y, gap, shift), Buffer(T * k, H, gt, gap=gap,
                                                                                          shift=shift)
    dw = torch.full((T, k), float("nan"), device=device())
    mp.combine_rows_backward(D.view, Y.view, position, w.to(device()), G.view, dw)
    torch.cuda.synchronize()
    assert G.outside_untouched()
    before = torch.as_strided(G.before, G.view.shape, G.view.stride(), G.view.storage_offset())
    got = set()
    exact_w, size_w = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        for s in range(k):
            p = int(position[t, s])
            if p < 0:
                continue
            got.add(p)
            v = float(w[t, s]) * d[t].double()
            bound = U32 * v.abs()
            assert_within(G.view[p], v, bound + HALF_STEP[gt] * (v.abs() + bound) + TINY[gt], f"dY[{p}]")
            exact_w[t, s] = (d[t].double() * y[p].double()).sum()
            size_w[t, s] = (d[t].double() * y[p].double()).abs().sum()
    assert_within(dw, exact_w, ((H + 63) // 64 + 16) * U32 * 1.01 * size_w, "dweights")
    for p in range(T * k):
        if p not in got:
            assert torch.equal(G.view[p], before[p])
    # without the weights' gradient Y is not needed
    again = Buffer(T * k, H, gt, gap=gap, shift=shift)
    mp.combine_rows_backward(D.view, None, position, w.to(device()), again.view)
    torch.cuda.synchronize()
    assert torch.equal(again.flat, G.flat)


def test_rows_gradients_against_differences():
    """The backward entry points are the derivative of the forward ones: a
    loss through gather and combine, both linear in x and in the weights, at
    two points."""
    dev = device()
    g = torch.Generator().manual_seed(4)
    T, k, E, H = 12, 3, 5, 33
    ids = make_ids(T, k, E, 8, drop=0.2)
    order, position, offsets = mp.route(ids.to(dev), E)
    x, w = torch.randn(T, H, generator=g).to(dev), torch.rand(T, k, generator=g).to(dev)
    c = torch.randn(T, H, generator=g).to(dev)

    def forward(x, w):
        rows = torch.zeros(T * k, H, device=dev)
        mp.gather_rows(x, order, rows, top_k=k)
        out = torch.empty(T, H, device=dev)
        mp.combine_rows(rows, position, out, weights=w)
        return rows, float((out.double() * c.double()).sum())

    rows, loss = forward(x, w)
    dy, dw = torch.zeros(T * k, H, device=dev), torch.empty(T, k, device=dev)
    mp.combine_rows_backward(c, rows, position, w, dy, dw)
    dx = torch.empty(T, H, device=dev)
    mp.combine_rows(dy, position, dx)
    ex, ew = torch.randn(T, H, generator=g).to(dev), torch.randn(T, k, generator=g).to(dev)
    size = float((c.abs().double() * 30).sum())
    # FP32 sums of values of size ~1..30: 1e-6 of the sum of magnitudes covers the forwards' rounding
    assert abs(forward(x + ex, w)[1] - loss - float((dx.double() * ex.double()).sum())) < 1e-6 * size
    assert abs(forward(x, w + ew)[1] - loss - float((dw.double() * ew.double()).sum())) < 1e-6 * size


# ---- grouped products -------------------------------------------------------

SIZES = [([5], 5), ([0, 0, 0], 4), ([3, 0, 64, 1, 130, 0], 200), ([1] * 70, 70), ([0] * 99 + [33], 40),
         ([64, 64], 128), ([300, 1, 2], 303)]


def check_grouped(sizes, R, N, K, dtype, col, alpha=1.0, beta=0.0, gap=0, shift=0, seed=1):
    dev = device()
    g = torch.Generator().manual_seed(seed + R + N + K)
    G = len(sizes)
    a = torch.randn(R, K, generator=g).to(dtype)
    b = torch.randn(G, K, N, generator=g).to(dtype)
    c = torch.randn(R, N, generator=g)
    if beta == 0.0:
        c.fill_(float("nan"))
    A, C = Buffer(R, K, dtype, a, gap, shift), Buffer(R, N, torch.float32, c, gap, shift)
    stored = b.transpose(1, 2).reshape(G * N, K) if col else b.reshape(G * K, N)
    B = Buffer(*stored.shape, dtype, stored, gap, shift)
    rows = N if col else K
    ld = B.view.stride(0)
    Bv = torch.as_strided(B.flat, (G, rows, stored.shape[1]), (rows * ld, ld, 1), B.view.storage_offset())
    Bv = Bv.transpose(1, 2) if col else Bv
    mp.gemm_grouped(A.view, Bv, C.view, offsets_of(sizes), alpha, beta)
    torch.cuda.synchronize()
    assert C.outside_untouched()
    lo = 0
    for e, n in enumerate(sizes):
        p = alpha * (a[lo:lo + n].double() @ b[e].double())
        mag = abs(alpha) * (a[lo:lo + n].double().abs() @ b[e].double().abs())
        if beta != 0.0:
            p, mag = p + beta * c[lo:lo + n].double(), mag + (beta * c[lo:lo + n].double()).abs()
        assert_within(C.view[lo:lo + n], p, (K + 2) * U32 * mag + 1e-40, f"group {e}")
        lo += n
    before = torch.as_strided(C.before, C.view.shape, C.view.stride(), C.view.storage_offset())
    assert torch.equal(C.view[lo:].view(torch.int32), before[lo:].view(torch.int32))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("col", [False, True])
@pytest.mark.parametrize("sizes,R", SIZES)
def test_grouped_sizes(dtype, col, sizes, R):
    check_grouped(sizes, R, 72, 144, dtype, col)


@pytest.mark.parametrize("col", [False, True])
@pytest.mark.parametrize("N,K,gap,shift", [(1, 1, 0, 0), (9, 7, 1, 1), (130, 65, 0, 0), (200, 333, 3, 1), (64, 1024, 0, 0)])
def test_grouped_shapes(col, N, K, gap, shift):
    check_grouped([7, 0, 70, 1], 90, N, K, torch.bfloat16, col, gap=gap, shift=shift)
    check_grouped([7, 0, 70, 1], 90, N, K, torch.float16, col, alpha=1.5, beta=-0.5, gap=gap, shift=shift)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("col", [False, True])
def test_grouped_every_tile_size(dtype, col):
    """Sizes at which each tile size and the narrow kernel are chosen, with
    ragged edges in every direction, C in whole lines and not."""
    check_grouped([1, 700, 0, 1299, 490], 2500, 1100, 77, dtype, col)
    check_grouped([300, 700, 0, 1299, 190], 2500, 2048, 530, dtype, col)
    check_grouped([300, 700, 0, 1299, 190], 2500, 2041, 530, dtype, col)
    check_grouped([230] * 13, 3000, 800, 300, dtype, col, gap=1)
    check_grouped([700, 900, 0, 899], 2500, 2048, 40, dtype, col)
    check_grouped([4000, 4900], 9000, 1024, 69, dtype, col)
    check_grouped([60] * 20, 1200, 1100, 100, dtype, col)
    check_grouped([9] * 70, 630, 515, 100, dtype, col)
    check_grouped([2] * 90, 180, 1030, 100, dtype, col)
    check_grouped([1, 4000, 0, 5, 4901], 9000, 1100, 69, dtype, col, beta=0.5)
    check_grouped([1, 9, 0, 16, 17], 50, 300, 1003, dtype, col, alpha=0.5, beta=2.0, gap=1, shift=1)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("K", [8, 24, 64, 100, 136])
@pytest.mark.parametrize("N", [5, 8, 13, 130, 257])
def test_grouped_edges_of_stored_rows(dtype, K, N):
    """Odd widths of operands stored along M and N, tightly packed at the end
    of their buffers, with K tiles that end at and beside the last row: the
    values behind a row are NaN where the sentinels are, and none of them may
    reach C."""
    dev = device()
    g = torch.Generator().manual_seed(K * N)
    a = torch.randn(K, N, generator=g).to(dtype)     # stored rows of the wgrad's A: K tokens x N
    b = torch.randn(K, 19, generator=g).to(dtype)
    flat = torch.full((K * N + 64,), float("nan"), dtype=dtype, device=dev)
    flat[:K * N] = a.reshape(-1).to(dev)
    A = flat[:K * N].view(K, N)
    out = torch.empty(2, N, 19, device=dev)
    sizes = [K - 5, 5]
    mp.gemm_grouped_wgrad(A.t(), b.to(dev), out, offsets_of(sizes))
    out2 = torch.empty(2, 19, N, device=dev)
    mp.gemm_grouped_wgrad(b.to(dev).t(), A, out2, offsets_of(sizes))
    x = torch.randn(70, K, generator=g).to(dtype)
    out3 = torch.empty(70, N, device=dev)
    mp.gemm_grouped(x.to(dev), A.unsqueeze(0), out3, offsets_of([70]))
    torch.cuda.synchronize()
    lo = 0
    for e, n in enumerate(sizes):
        u, v = a[lo:lo + n].double(), b[lo:lo + n].double()
        bound = (n + 2) * U32 * (u.abs().t() @ v.abs()) + 1e-40
        assert_within(out[e], u.t() @ v, bound, "wgrad")
        assert_within(out2[e], v.t() @ u, bound.t(), "wgrad, operands exchanged")
        lo += n
    assert_within(out3, x.double() @ a.double(), (K + 2) * U32 * (x.double().abs() @ a.double().abs()), "rows")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_wgrad_every_tile_size(dtype):
    check_wgrad([100, 0, 37, 1], 140, 900, 1100, dtype)
    check_wgrad([30, 7, 0], 40, 2200, 3300, dtype, beta=0.5)
    check_wgrad([30, 7, 0], 40, 2048, 2048, dtype)
    check_wgrad([700, 400], 1100, 2000, 2048, dtype)
    check_wgrad([700, 400], 1100, 2001, 2043, dtype)
    check_wgrad([70, 0, 400], 470, 2300, 4096, dtype)
    check_wgrad([70, 0, 400], 470, 2300, 4097, dtype, beta=1.0)


def test_grouped_scalars_and_empty():
    check_grouped([3, 4], 8, 20, 0, torch.float16, True, beta=0.5)
    check_grouped([3, 4], 8, 20, 0, torch.float16, False)
    check_grouped([0], 0, 20, 8, torch.float16, False)
    # alpha == 0 reads neither A nor B
    dev = device()
    nan = torch.full((6, 40), float("nan"), dtype=torch.float16, device=dev)
    c = torch.ones(6, 24, device=dev)
    mp.gemm_grouped(nan, nan[:2, :1].expand(2, 24).reshape(2, 1, 24).repeat(1, 40, 1), c, offsets_of([2, 3]), 0.0, 2.0)
    assert (c[:5] == 2).all() and (c[5] == 1).all()


@pytest.mark.parametrize("bad", [[0, 9, 3, 12, 500], [-7, 4, 4, 1 << 30, -1], [12, 8, 4, 0, 0], [0, 12, 0, 12, 0]])
def test_grouped_wrong_offsets_stay_inside(bad):
    dev = device()
    off = torch.tensor(bad, dtype=torch.int32, device=dev)
    a, b = torch.randn(12, 40).to(torch.float16).to(dev), torch.randn(4, 40, 24).to(torch.float16).to(dev)
    C = Buffer(12, 24, torch.float32)
    mp.gemm_grouped(a, b, C.view, off)
    W = Buffer(4 * 40, 24, torch.float32)
    mp.gemm_grouped_wgrad(a.t(), torch.randn(12, 24).to(torch.float16).to(dev), W.view.view(4, 40, 24), off)
    torch.cuda.synchronize()
    assert C.outside_untouched() and W.outside_untouched()


def check_wgrad(sizes, R, M, N, dtype, alpha=1.0, beta=0.0, gap=0, shift=0):
    g = torch.Generator().manual_seed(R + M + N)
    G = len(sizes)
    a, b = torch.randn(R, M, generator=g).to(dtype), torch.randn(R, N, generator=g).to(dtype)
    c = torch.randn(G * M, N, generator=g)
    if beta == 0.0:
        c.fill_(float("nan"))
    A, B, C = (Buffer(R, M, dtype, a, gap, shift), Buffer(R, N, dtype, b, gap, shift),
               Buffer(G * M, N, torch.float32, c, gap, shift))
    ld = C.view.stride(0)
    Cv = torch.as_strided(C.flat, (G, M, N), (M * ld, ld, 1), C.view.storage_offset())
    mp.gemm_grouped_wgrad(A.view.t(), B.view, Cv, offsets_of(sizes), alpha, beta)
    torch.cuda.synchronize()
    assert C.outside_untouched()
    lo = 0
    for e, n in enumerate(sizes):
        x, y = a[lo:lo + n].double(), b[lo:lo + n].double()
        p, mag = alpha * (x.t() @ y), abs(alpha) * (x.abs().t() @ y.abs())
        if beta != 0.0:
            old = beta * c[e * M:(e + 1) * M].double()
            p, mag = p + old, mag + old.abs()
        assert_within(Cv[e], p, (n + 2) * U32 * mag + 1e-40, f"group {e}")
        lo += n


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("sizes,R", SIZES)
def test_wgrad_sizes(dtype, sizes, R):
    check_wgrad(sizes, R, 72, 40, dtype)


@pytest.mark.parametrize("M,N,gap,shift", [(1, 1, 0, 0), (9, 7, 1, 1), (130, 65, 0, 0), (200, 333, 3, 1), (256, 128, 0, 0)])
def test_wgrad_shapes(M, N, gap, shift):
    check_wgrad([7, 0, 70, 1, 200], 290, M, N, torch.bfloat16, gap=gap, shift=shift)
    check_wgrad([7, 0, 70, 1, 200], 290, M, N, torch.float16, alpha=0.5, beta=1.0, gap=gap, shift=shift)


def test_wgrad_no_rows():
    check_wgrad([0, 0], 0, 20, 30, torch.float16)
    check_wgrad([0, 0], 0, 20, 30, torch.float16, beta=0.5)


def test_expert_layer_forward_and_backward():
    """route, gather, grouped product, combine and their gradients, as a
    training step runs them, against the layer in 64 bits on the CPU (the
    gradient of the loss <out, c> by x, the experts' and the slots' weights).
    What is rounded to bfloat16 on the way is rounded in the reference too, so
    only FP32 roundings differ, each sum of n products at most (n + 2)*u of its
    magnitudes: the longest way is a slot weight's gradient, a product over H
    = 96 and a dot product of at most 17 additions, 115*u in all, under 1e-5 =
    168*u of the magnitudes."""
    dev = device()
    g = torch.Generator().manual_seed(21)
    T, k, E, H, N = 45, 3, 7, 96, 56
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    w = torch.randn(E, N, H, generator=g).to(torch.bfloat16)
    slots = torch.rand(T, k, generator=g)
    c = torch.randn(T, N, generator=g).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    ids[3, 1], ids[9] = -1, E
    R = T * k
    order, position, offsets = mp.route(ids.to(dev), E)
    rows = torch.zeros(R, H, dtype=torch.bfloat16, device=dev)
    y, out = torch.zeros(R, N, device=dev), torch.empty(T, N, device=dev)
    wd, sd, cd = w.to(dev), slots.to(dev), c.to(dev)
    mp.gather_rows(x.to(dev), order, rows, top_k=k)
    mp.gemm_grouped(rows, wd.mT, y, offsets)
    mp.combine_rows(y, position, out, weights=sd)
    dy, dslots = torch.zeros(R, N, dtype=torch.bfloat16, device=dev), torch.empty(T, k, device=dev)
    mp.combine_rows_backward(cd, y, position, sd, dy, dslots)
    drows, dw, dx = torch.zeros(R, H, device=dev), torch.empty(E, N, H, device=dev), torch.empty(T, H, device=dev)
    mp.gemm_grouped(dy, wd, drows, offsets)
    mp.gemm_grouped_wgrad(dy.t(), rows, dw, offsets)
    mp.combine_rows(drows, position, dx)
    torch.cuda.synchronize()
    zero = lambda *s: torch.zeros(s, dtype=torch.float64)  # noqa: E731
    want = {n: [zero(*s), zero(*s)] for n, s in
            (("out", (T, N)), ("dslots", (T, k)), ("dx", (T, H)), ("dw", (E, N, H)))}

    def add(name, at, value, size):
        want[name][0][at] += value
        want[name][1][at] += size

    for t in range(T):
        for s in range(k):
            e = int(ids[t, s])
            if not 0 <= e < E:
                continue
            xt, we, ct, ws = x[t].double(), w[e].double(), c[t].double(), float(slots[t, s])
            p, mag = we @ xt, we.abs() @ xt.abs()
            gy = (slots[t, s] * c[t].float()).to(torch.bfloat16).double()  # one FP32 product, rounded
            add("out", t, ws * p, ws * mag)
            add("dslots", (t, s), (ct * p).sum(), (ct.abs() * mag).sum())
            add("dx", t, we.t() @ gy, we.abs().t() @ gy.abs())
            add("dw", e, torch.outer(gy, xt), torch.outer(gy, xt).abs())
    for name, got in (("out", out), ("dslots", dslots), ("dx", dx), ("dw", dw)):
        assert_within(got, want[name][0], 1e-5 * want[name][1], name)


def test_grouped_graph_and_stream():
    dev = device()
    a, b = torch.randn(64, 128).to(torch.bfloat16).to(dev), torch.randn(8, 128, 96).to(torch.bfloat16).to(dev)
    off = offsets_of([8] * 8)
    eager = torch.empty(64, 96, device=dev)
    mp.gemm_grouped(a, b, eager, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty(64, 96, device=dev)
    side.wait_stream(torch.cuda.current_stream())
    mp.gemm_grouped(a, b, out, off, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    dw = torch.empty(8, 128, 96, device=dev)
    mp.gemm_grouped_wgrad(a.t(), eager.to(torch.bfloat16), dw, off)
    eager_dw = dw.clone()
    gy = eager.to(torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mp.gemm_grouped(a, b, out, off)
        mp.gemm_grouped_wgrad(a.t(), gy, dw, off)
    for _ in range(3):
        out.zero_()
        dw.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(dw, eager_dw)
