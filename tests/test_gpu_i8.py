"""GPU: rows to 8-bit codes and the product of codes, against their
definitions in 64 bits.

Bounds (u = 2^-24, half a step of FP32; h the output type's half step):
codes and scales are equal to the definition's, which is exact.  The product
is the exact sum s, rounded (u), times two scales (2u), so 3u + 3u^2 + ... <
3.01u of |s*sa*sw|; the bias adds u of the result; the output type h of it (or
half its smallest step below the normal numbers)."""
import pytest
import torch

import dense_mixed_precision_amd as mp
from tests.gpu_util import device
from tests.ops_util import HALF_STEP, TINY, U32, Buffer, assert_within, offsets_of, order_by_expert

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16, torch.float32]


def codes_of(x):
    """(codes, scale) by definition, on the CPU: exact quotients (64 bits hold
    127*x; no quotient of 24-bit values is nearer than 2^-33 to a middle
    without being one), scale rounded to FP32 once."""
    x = x.cpu().double()
    top = x.abs().amax(1) if x.shape[1] else x.new_zeros(x.shape[0])
    bad = ~torch.isfinite(x).all(1)
    safe = torch.where((top > 0) & ~bad, top, 1.0)
    codes = torch.round(torch.where(bad[:, None], 0.0, 127.0 * x) / safe[:, None])
    scale = torch.where(bad, float("nan"), top / 127.0)
    return codes.to(torch.int8), scale.float()


def check_quantize(x, dtype, gap=0, shift=0, order=None, top_k=1, rows=None):
    T, H = x.shape
    R = T if order is None else len(order)
    X = Buffer(T, H, dtype, x.to(dtype), gap, shift)
    Q = Buffer(R, H, torch.int8, gap=gap, shift=shift)
    S = Buffer(1, R, torch.float32)
    od = None if order is None else torch.tensor(order, dtype=torch.int32, device=device())
    mp.quantize_rows(X.view, Q.view, S.view.reshape(-1) if R else S.flat[:0], order=od, top_k=top_k)
    torch.cuda.synchronize()
    codes, scale = codes_of(X.view)
    want_q, want_s = Q.before.clone(), S.before.clone()
    wq = torch.as_strided(want_q, Q.view.shape, Q.view.stride(), Q.view.storage_offset())
    ws = torch.as_strided(want_s, (R,), (1,), S.view.storage_offset())
    for p in range(R):
        src = p if order is None else (order[p] // top_k if 0 <= order[p] < T * top_k else -1)
        if src >= 0:
            wq[p] = codes[src].to(device())
            ws[p] = scale[src]
    assert torch.equal(Q.flat, want_q)
    assert torch.equal(S.flat.view(torch.int32), want_s.view(torch.int32)) or (
        torch.equal(torch.isnan(S.flat), torch.isnan(want_s)) and
        torch.equal(torch.nan_to_num(S.flat), torch.nan_to_num(want_s)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,gap,shift", [(1, 1, 0, 0), (3, 7, 1, 1), (5, 64, 0, 0), (2, 2048, 0, 0), (4, 2049, 3, 1),
                                           (3, 8192, 0, 0), (2, 20000, 5, 1), (130, 96, 0, 0), (4, 0, 0, 0),
                                           (17, 128, 0, 0), (18, 256, 1, 1), (17, 257, 0, 0), (8200, 300, 1, 1),
                                           (8192, 1024, 0, 0), (2050, 1025, 0, 1), (2049, 4096, 0, 0)])
def test_quantize_sizes(dtype, T, H, gap, shift):
    g = torch.Generator().manual_seed(T * 7919 + H)
    check_quantize(torch.randn(T, H, generator=g) * torch.exp(2 * torch.randn(T, 1, generator=g)), dtype, gap, shift)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_middles_and_extremes(dtype):
    big = torch.finfo(dtype).max
    small = torch.finfo(dtype).tiny
    step = small * torch.finfo(dtype).eps  # the smallest number
    rows = torch.zeros(12, 256, dtype=torch.float64)
    rows[0] = torch.arange(256) - 127.5          # halves: with the maximum 127 every value is a middle
    rows[0, 255] = 127.0
    rows[1] = (torch.arange(256) - 128) / 256.0
    rows[2, 5] = -big
    rows[2, 6] = big / 2
    rows[3] = step * torch.arange(256)            # below the normal numbers
    rows[4, 0] = step
    rows[6, 3] = float("inf")
    rows[7, 9] = float("nan")
    rows[8, 9], rows[8, 10] = float("-inf"), float("nan")
    rows[9] = small * (torch.arange(256) - 128)
    rows[10] = -0.0
    rows[11] = torch.linspace(-1, 1, 256) * big / 3
    check_quantize(rows, dtype)


def test_quantize_next_to_a_middle():
    """FP32 values one step beside the middle of two codes."""
    g = torch.Generator().manual_seed(5)
    top = torch.rand(64, 1, generator=g) + 1.0
    n = torch.randint(0, 126, (64, 255), generator=g)
    mid = ((n + 0.5) * (top.double() / 127.0)).float()
    way = torch.randint(-1, 2, (64, 255), generator=g)
    x = torch.where(way == 0, mid, torch.nextafter(mid, torch.where(way > 0, torch.inf, 0.0)))
    check_quantize(torch.cat([x, top], 1), torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_by_order(dtype):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(9, 70, generator=g)
    # the same row twice, absent rows, indices outside
    check_quantize(x, dtype, gap=2, order=[4, 17, 0, 1, 1, -1, 16, 18, 1 << 30, -5], top_k=2)
    check_quantize(x[:0], dtype, order=[0, -1, 3])


@pytest.mark.parametrize("dtype,T,k,H,gap,shift", [(torch.bfloat16, 6000, 3, 2051, 1, 1), (torch.float32, 4100, 2, 2304, 0, 0),
                                                   (torch.float16, 700, 9, 6000, 8, 0)])
def test_quantize_many_rows(dtype, T, k, H, gap, shift):
    """Rows enough for the way by tokens, also where the order is no
    permutation: pairs absent, twice, outside."""
    g = torch.Generator().manual_seed(H)
    R = T * k
    order = torch.randperm(R, generator=g, dtype=torch.int64).to(torch.int32)
    order[5], order[R // 2], order[R // 3] = int(order[0]), int(order[0]), int(order[1])
    order[7], order[8], order[9], order[10:400] = R, -2, (1 << 31) - 1, -1
    assert mp.mpgemm_rows_workspace(mp.MPGEMM_T_F32 if dtype == torch.float32 else 0, T, H, R, k) > 0
    x = torch.randn(T, H, generator=g)
    x[3, 5], x[4] = float("inf"), 0.0
    X = Buffer(T, H, dtype, x.to(dtype), gap, shift)
    Q, S = Buffer(R, H, torch.int8, gap=gap, shift=shift), Buffer(1, R, torch.float32)
    mp.quantize_rows(X.view, Q.view, S.view.reshape(-1), order=order.to(device()), top_k=k)
    torch.cuda.synchronize()
    codes, scale = codes_of(X.view)
    there = ((order >= 0) & (order < R)).nonzero().reshape(-1)
    src = (order[there] // k).long()
    wq = torch.as_strided(Q.before, Q.view.shape, Q.view.stride(), Q.view.storage_offset()).cpu().clone()
    ws = torch.as_strided(S.before, (R,), (1,), S.view.storage_offset()).cpu().clone()
    wq[there], ws[there] = codes[src], scale[src]
    got_s = S.view.reshape(-1).cpu()
    assert torch.equal(Q.view.cpu(), wq) and Q.outside_untouched() and S.outside_untouched()
    assert torch.equal(torch.isnan(got_s), torch.isnan(ws))
    assert torch.equal(torch.nan_to_num(got_s), torch.nan_to_num(ws))


def test_quantize_another_stream_and_a_graph():
    x = torch.randn(16, 512, device=device())
    q = torch.zeros(16, 512, dtype=torch.int8, device=device())
    s = torch.zeros(16, device=device())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mp.quantize_rows(x, q, s, stream=side)
    torch.cuda.synchronize()
    codes, scale = codes_of(x)
    assert torch.equal(q.cpu(), codes) and torch.equal(s.cpu(), scale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mp.quantize_rows(x, q, s)
    for r in range(3):
        x.copy_(torch.randn(16, 512, device=device()) * (r + 1))
        q.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        codes, scale = codes_of(x)
        assert torch.equal(q.cpu(), codes) and torch.equal(s.cpu(), scale)


# ---- products ---------------------------------------------------------------

def make_i8(M, N, K, G, seed, extremes=False):
    g = torch.Generator().manual_seed(seed)
    a = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8)
    w = torch.randint(-127, 128, (G, N, K), generator=g, dtype=torch.int8)
    if extremes:
        a.fill_(-128)
        w.fill_(-128)
    sa = torch.rand(M, generator=g) + 0.01
    sw = (torch.rand(G, N, generator=g) + 0.01) / 64
    bias = 100 * torch.randn(G, N, generator=g)
    return a, w, sa, sw, bias


def check_i8(M, N, K, dtype, sizes=None, gap=0, shift=0, bias=True, seed=1, extremes=False):
    G = 1 if sizes is None else len(sizes)
    a, w, sa, sw, b = make_i8(M, N, K, G, seed, extremes)
    if dtype == torch.float16:
        sw = sw / (16 * max(K, 1))   # keep the products within FP16
    A = Buffer(M, K, torch.int8, a, gap, shift)
    W = Buffer(G * N, K, torch.int8, w.reshape(G * N, K), gap, shift)
    C = Buffer(M, N, dtype, gap=gap, shift=shift)
    dev = device()
    wv = torch.as_strided(W.flat, (G, N, K), (N * W.view.stride(0), W.view.stride(0), 1), W.view.storage_offset())
    off = None if sizes is None else offsets_of(sizes)
    bd = b.to(dev) if bias else None
    if sizes is None:
        wv = wv[0]
        mp.gemm_i8(A.view, wv.t(), C.view, sa.to(dev), sw[0].to(dev), bias=bd[0] if bias else None)
    else:
        mp.gemm_i8(A.view, wv.transpose(1, 2), C.view, sa.to(dev), sw.to(dev), bias=bd, offsets=off)
    torch.cuda.synchronize()
    assert C.outside_untouched()
    ends = [0, M] if sizes is None else [0] + torch.tensor(sizes).cumsum(0).tolist()
    for e in range(G):
        lo, hi = ends[e], ends[e + 1]
        p = (a[lo:hi].double() @ w[e].double().t()) * sa[lo:hi, None].double() * sw[e].double()
        v = p + b[e].double() if bias else p
        bound = 3.01 * U32 * p.abs() + (1.01 * U32 if bias else 0) * v.abs()
        bound = bound + HALF_STEP[dtype] * (v.abs() + bound) + TINY[dtype]
        assert_within(C.view[lo:hi], v, bound, f"{M}x{N}x{K} group {e}")
    if sizes is not None and ends[-1] < M:
        before = torch.as_strided(C.before, C.view.shape, C.view.stride(), C.view.storage_offset())
        assert torch.equal(C.view[ends[-1]:], before[ends[-1]:])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 16, 64), (2, 3, 5), (16, 16, 16), (17, 33, 100), (64, 64, 128),
                                   (65, 63, 129), (100, 90, 77), (128, 256, 512), (7, 1000, 617), (130, 257, 1039)])
def test_i8_sizes(dtype, M, N, K):
    check_i8(M, N, K, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K,gap", [(1500, 1400, 200, 0), (2600, 4100, 141, 0), (2570, 4353, 300, 3),
                                       (16, 4100, 1000, 0), (12, 300, 5001, 1), (2040, 4000, 600, 0), (1700, 2000, 700, 1),
                                       (1200, 4400, 130, 1), (1100, 1101, 200, 0), (500, 1000, 333, 2), (300, 1000, 400, 0),
                                       (16, 16400, 520, 0)])
def test_i8_every_tile_size(dtype, M, N, K, gap):
    """Sizes at which each tile size and the narrow kernel's two forms are
    chosen, with ragged edges in every direction."""
    check_i8(M, N, K, dtype, gap=gap)


def test_i8_groups_every_tile_size():
    check_i8(2500, 1100, 200, torch.bfloat16, sizes=[1, 700, 0, 1299, 490])
    check_i8(9000, 1100, 133, torch.float32, sizes=[1, 4000, 0, 5, 4901], gap=1)
    check_i8(2500, 2040, 600, torch.float32, sizes=[300, 700, 0, 1299, 190])
    check_i8(800, 1030, 300, torch.float16, sizes=[8] * 99 + [7])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gap,shift", [(0, 1), (1, 0), (3, 3), (16, 0)])
def test_i8_alignments(dtype, gap, shift):
    check_i8(70, 83, 300, dtype, gap=gap, shift=shift, seed=gap + 8 * shift)


@pytest.mark.parametrize("K", [1, 15, 16, 17, 31, 54, 59, 127, 128, 129, 143, 255, 257, 271])
@pytest.mark.parametrize("M,N", [(3, 20), (40, 50), (100, 520), (600, 2000)])
def test_i8_ends_of_rows(M, N, K):
    """Rows whose last vector straddles K, in every kernel, tightly packed."""
    check_i8(M, N, K, torch.float32, seed=K)
    check_i8(M, N, K, torch.bfloat16, gap=5, shift=1, bias=False, seed=K)


@pytest.mark.parametrize("M,N,K", [(5, 9, 0), (0, 9, 5), (5, 0, 5)])
def test_i8_empty(M, N, K):
    check_i8(M, N, K, torch.float32)


def test_i8_views_of_weights():
    """Weights as a user may hold them: one row, one column, one value, a slice
    of wider rows, and what is refused."""
    dev = device()
    g = torch.Generator().manual_seed(6)
    big = torch.randint(-9, 10, (40, 64), generator=g, dtype=torch.int8).to(dev)
    a = torch.randint(-9, 10, (7, 64), generator=g, dtype=torch.int8).to(dev)

    def run(a, w):  # w: K x N view
        out = torch.empty(a.shape[0], w.shape[1], device=dev)
        one = torch.ones(64, device=dev)
        mp.gemm_i8(a, w, out, one[:a.shape[0]], one[:w.shape[1]])
        assert torch.equal(out.double().cpu(), a.double().cpu() @ w.double().cpu())

    run(a, big.t())
    run(a, big[:1].t())
    run(a, big[3].view(64, 1))
    run(a[:, :1].contiguous(), big[:, :1].t())
    run(a[:, :1].contiguous(), big[:1, :1])
    run(a[:, :33].contiguous(), big[5:25, 10:43].t())
    run(a[:, :33], big[5:25, 10:43].t())
    run(a[:, :0].contiguous(), big[:, :0].t())
    for bad in (big.t().contiguous(), big[:, ::2].t(), big.float().t(), big[:, :1].expand(40, 64).t(), big.cpu().t(), None):
        with pytest.raises((ValueError, TypeError)):
            mp.gemm_i8(a, bad, torch.empty(7, 40, device=dev), torch.ones(7, device=dev), torch.ones(40, device=dev))


def test_i8_largest_sum():
    """Every code -128 at the largest K: the sum is 131071 * 2^14."""
    check_i8(3, 18, mp.MPGEMM_I8_MAX_K, torch.float32, extremes=True, bias=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes,M", [([5], 5), ([0, 0, 0], 4), ([3, 0, 64, 1, 130, 0], 200), ([1] * 70, 70),
                                     ([0] * 99 + [33], 40), ([64, 64], 128), ([300, 1, 2], 303)])
def test_i8_groups(dtype, sizes, M):
    check_i8(M, 72, 144, dtype, sizes=sizes)


def test_i8_groups_ragged_and_misaligned():
    check_i8(50, 37, 93, torch.float16, sizes=[7, 0, 20, 11], gap=1, shift=1)


def test_i8_nan_scale_reaches_its_row_only():
    a, w, sa, sw, _ = make_i8(5, 20, 64, 1, 9)
    sa[2] = float("nan")
    out = torch.zeros(5, 20, device=device())
    mp.gemm_i8(a.to(device()), w[0].to(device()).t(), out, sa.to(device()), sw[0].to(device()))
    nan = torch.isnan(out).cpu()
    assert nan[2].all() and not nan[[0, 1, 3, 4]].any()


@pytest.mark.parametrize("bad", [[0, 9, 3, 12, 500], [-7, 4, 4, 1 << 30, -1], [12, 8, 4, 0, 0], [0, 12, 0, 12, 0]])
def test_i8_wrong_offsets_stay_inside(bad):
    """Offsets that are no partition: some result, nothing outside C."""
    a, w, sa, sw, _ = make_i8(12, 20, 64, 4, 9)
    C = Buffer(12, 20, torch.float32)
    mp.gemm_i8(a.to(device()), w.to(device()).transpose(1, 2), C.view, sa.to(device()), sw.to(device()),
               offsets=torch.tensor(bad, dtype=torch.int32, device=device()))
    torch.cuda.synchronize()
    assert C.outside_untouched()


def test_experts_in_8_bits_end_to_end():
    """route, quantize in expert order, product, combine: as a serving layer
    runs them, against the same steps in 64 bits on the codes."""
    dev = device()
    g = torch.Generator().manual_seed(11)
    T, k, E, H, N = 37, 3, 6, 200, 90
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    ids[5] = -1
    weights = torch.rand(T, k, generator=g)
    w = torch.randint(-127, 128, (E, N, H), generator=g, dtype=torch.int8)
    sw = torch.rand(E, N, generator=g) / 100
    order, position, offsets = mp.route(ids.to(dev), E)
    R = T * k
    q = torch.zeros(R, H, dtype=torch.int8, device=dev)
    s = torch.zeros(R, device=dev)
    y = torch.zeros(R, N, dtype=torch.bfloat16, device=dev)
    out = torch.empty(T, N, device=dev)
    mp.quantize_rows(x.to(dev), q, s, order=order, top_k=k)
    mp.gemm_i8(q, w.to(dev).transpose(1, 2), y, s, sw.to(dev), offsets=offsets)
    mp.combine_rows(y, position, out, weights=weights.to(dev))
    torch.cuda.synchronize()
    codes, scale = codes_of(x)
    exact, bound = torch.zeros(T, N, dtype=torch.float64), torch.zeros(T, N, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e < 0:
                continue
            p = (codes[t].double() @ w[e].double().t()) * float(scale[t]) * sw[e].double() * float(weights[t, j])
            exact[t] += p
            # product 3u, its rounding to bfloat16 2^-8, the weighted sum u per slot
            bound[t] += (3.01 * U32 + 2.0 ** -8 * 1.001 + (k + 1) * U32) * p.abs()
    assert_within(out, exact, bound + 1e-30, "experts in 8 bits")
    want = order_by_expert(ids, E)
    assert order.tolist() == want[0] and offsets.tolist() == want[2]
