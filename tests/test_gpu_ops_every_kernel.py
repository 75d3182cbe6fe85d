"""GPU: every kernel of the operators' products where it can go wrong, each
asked for by a query: ends of rows at every kind of K, odd widths, shifted and
gapped operands, empty and foreign groups, offsets that are no partition; and
every combination of types of the rows' gradients.

Values are small whole numbers and scales powers of two, so that every product
and sum is exact in FP32 whatever its order, and results are compared for
equality with the definition in 64 bits, rounded as stated: sums stay below
1031 * 127^2 < 2^24, those of 16-bit values below 640 * 4 * 4 * 2 + 8 < 2^24."""
import pytest
import torch

import dense_mixed_precision_amd as mp
from tests import ops_kernels as ok
from tests.gpu_util import device
from tests.ops_util import Buffer

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
NAN = float("nan")


def whole(gen, most, *shape, dtype):
    return torch.randint(-most, most + 1, shape, generator=gen, device=device(), dtype=torch.int32).to(dtype)


def powers(gen, low, high, *shape):
    return torch.exp2(torch.randint(low, high + 1, shape, generator=gen, device=device()).float())


def generator(*seed):
    return torch.Generator(device=device()).manual_seed(sum((i + 1) * s for i, s in enumerate(seed)))


def sizes_of(G, rows):
    """Group sizes of `rows` rows: an empty one, one of a single row."""
    if G == 2:
        return [rows - rows // 3, rows // 3]
    sizes = [rows // 3, 0, 1] + [0] * (G - 4)
    return sizes + [rows - sum(sizes)]


def ends_of(sizes, first):
    ends = [first]
    for n in sizes:
        ends.append(ends[-1] + n)
    return ends


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=device())


def matrices(buffer, G, rows, cols):
    """A Buffer of G * rows rows as G matrices."""
    ld = buffer.view.stride(0)
    return torch.as_strided(buffer.flat, (G, rows, cols), (rows * ld, ld, 1), buffer.view.storage_offset())


def same(got, want):
    """Equal, NaN at the same places."""
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(torch.where(nan, 0, got), torch.where(nan, 0, want))


def old(buffer):
    return torch.as_strided(buffer.before, buffer.view.shape, buffer.view.stride(), buffer.view.storage_offset())


# ---- 8-bit products ---------------------------------------------------------

# (C, gap, shift, with a bias): odd places, and rows on whole 128-byte lines
I8_FORMS = [(F32, 0, 0, True), (BF16, 5, 1, False), (F16, 16, 3, True)]


def i8_operands(M, N, K, G, C, gap, shift, bias):
    g = generator(M, N, K, G)
    A = Buffer(M, K, torch.int8, whole(g, 127, M, K, dtype=torch.int8), gap, shift)
    W = Buffer(G * N, K, torch.int8, whole(g, 127, G * N, K, dtype=torch.int8), gap, shift)
    sa, sb = powers(g, -12, -6, M), powers(g, -12, -6, G, N)
    b = whole(g, 50, G, N, dtype=F32) / 16 if bias else None
    return A, W, Buffer(M, N, C, gap=gap, shift=shift), sa, sb, b


def i8_rows(A, W, sa, sb, b, C):
    """64 bits hold the value whole; FP32, then the type of C."""
    v = (A.double() @ W.double().t()) * sa.double()[:, None] * sb.double()
    return (v if b is None else v + b.double()).float().to(C)


@pytest.mark.parametrize("kernel,K", [(k, K) for k, case in ok.I8.items() for K in case[2]])
@pytest.mark.parametrize("lines", [False, True])
def test_i8_ends_of_rows(kernel, K, lines):
    M, N, _ = ok.I8[kernel]
    if lines:
        N = (N + 63) // 64 * 64
    for C, gap, shift, bias in [(F32, 0, 0, False), (BF16, 0, 0, True)] if lines else I8_FORMS:
        assert ok.i8_kernel(0, M, N, K, gap) == kernel
        A, W, O, sa, sb, b = i8_operands(M, N, K, 1, C, gap, shift, bias)
        mp.gemm_i8(A.view, W.view.t(), O.view, sa, sb[0], bias=None if b is None else b[0])
        torch.cuda.synchronize()
        same(O.view, i8_rows(A.view, W.view, sa, sb[0], None if b is None else b[0], C))
        assert O.outside_untouched()


@pytest.mark.parametrize("kernel,K", [(k, K) for k, case in ok.I8_GROUPS.items() for K in case[3]])
def test_i8_groups(kernel, K):
    """Rows before the first group and behind the last keep what they hold;
    a scale that is NaN reaches its row or column alone."""
    G, M, N, _ = ok.I8_GROUPS[kernel]
    for C, gap, shift, bias in I8_FORMS:
        assert ok.i8_kernel(G, M, N, K, gap) == kernel
        A, W, O, sa, sb, b = i8_operands(M, N, K, G, C, gap, shift, bias)
        ends = ends_of(sizes_of(G, M - 11), 6)
        sa[:6], sa[ends[-1]:], sa[ends[1] - 1], sb[G - 1, N // 2] = NAN, NAN, NAN, NAN
        w = matrices(W, G, N, K)
        mp.gemm_i8(A.view, w.mT, O.view, sa, sb, bias=b, offsets=i32(ends))
        torch.cuda.synchronize()
        want = old(O).clone()
        for e in range(G):
            here = slice(ends[e], ends[e + 1])
            want[here] = i8_rows(A.view[here], w[e], sa[here], sb[e], None if b is None else b[e], C)
        same(O.view, want)
        assert O.outside_untouched()


def no_partition(G, R):
    """Offsets that are none, of G groups over R rows."""
    return [(x + [R] * G)[:G + 1] for x in ([0, R - 3, 3, R, 40 * R], [-7, 4, 4, 1 << 30, -1], [R, 8, 4, 0, 0],
                                            [0, R, 0, R, 0], [R + 9, R + 9, -1 << 31, R, 2])]


@pytest.mark.parametrize("kernel", list(ok.I8_GROUPS))
def test_i8_wrong_offsets_stay_inside(kernel):
    G, M, N, Ks = ok.I8_GROUPS[kernel]
    for ends in no_partition(G, M):
        A, W, O, sa, sb, b = i8_operands(M, N, Ks[-1], G, F32, 5, 1, True)
        mp.gemm_i8(A.view, matrices(W, G, N, Ks[-1]).mT, O.view, sa, sb, bias=b, offsets=i32(ends))
        torch.cuda.synchronize()
        assert O.outside_untouched()


# ---- grouped 16-bit products ------------------------------------------------

# (type, gap, shift, alpha, beta)
FORMS = [(F16, 0, 0, 1.0, 0.0), (BF16, 1, 1, 2.0, -0.5), (BF16, 8, 0, 1.0, 1.0)]


def grouped_operands(G, R, N, K, lb, dtype, gap, shift, beta):
    g = generator(G, R, N, K)
    A = Buffer(R, K, dtype, whole(g, 4, R, K, dtype=dtype), gap, shift)
    rows, cols = (N, K) if lb == ok.COL else (K, N)
    B = Buffer(G * rows, cols, dtype, whole(g, 4, G * rows, cols, dtype=dtype), gap, shift)
    C = Buffer(R, N, F32, whole(g, 8, R, N, dtype=F32) if beta else torch.full((R, N), NAN), gap, shift)
    b = matrices(B, G, rows, cols)
    return A, (b.mT if lb == ok.COL else b), C


@pytest.mark.parametrize("kernel,lb,K", [(k, lb, K) for (k, lb), case in ok.GROUPED.items() for K in case[3]])
def test_grouped_ends_of_rows(kernel, lb, K):
    """Rows of no group and the whole first group (rows and matrix) are NaN,
    which stays there."""
    G, R, N, _ = ok.GROUPED[kernel, lb]
    for dtype, gap, shift, alpha, beta in FORMS:
        if lb == ok.COL and K <= 1 and gap == 0:
            continue  # the bytes of a row-major matrix, and taken as one
        assert ok.grouped_kernel(lb, G, R, N, K, gap) == kernel
        A, B, C = grouped_operands(G, R, N, K, lb, dtype, gap, shift, beta)
        ends = ends_of(sizes_of(G, R - 11), 6)
        A.view[:ends[1]], A.view[ends[-1]:], B[0] = NAN, NAN, NAN
        mp.gemm_grouped(A.view, B, C.view, i32(ends), alpha, beta)
        torch.cuda.synchronize()
        want = old(C).clone()
        for e in range(G):
            here = slice(ends[e], ends[e + 1])
            v = alpha * (A.view[here].double() @ B[e].double())
            want[here] = (v + beta * want[here].double() if beta else v).float()
        same(C.view, want)
        assert C.outside_untouched()


@pytest.mark.parametrize("kernel,lb", list(ok.GROUPED))
def test_grouped_wrong_offsets_stay_inside(kernel, lb):
    G, R, N, Ks = ok.GROUPED[kernel, lb]
    for ends in no_partition(G, R):
        A, B, C = grouped_operands(G, R, N, Ks[-1], lb, BF16, 1, 1, 0.0)
        mp.gemm_grouped(A.view, B, C.view, i32(ends))
        torch.cuda.synchronize()
        assert C.outside_untouched()


@pytest.mark.parametrize("rows", [0, 1, 7, 8, 9, 63, 64, 65, 71, 127, 130])
@pytest.mark.parametrize("kernel", list(ok.WGRAD))
def test_wgrad_ends_of_groups(kernel, rows):
    """A group of every kind of length beside another; rows of no group are
    NaN, and the values behind a row the buffer's margins."""
    G, R, M, N = ok.WGRAD[kernel]
    for dtype, gap, shift, alpha, beta in FORMS:
        for n in (N, (N + 31) // 32 * 32):
            assert ok.wgrad_kernel(G, R, M, n, gap) == kernel
            g = generator(R, M, n, rows)
            A = Buffer(R, M, dtype, whole(g, 4, R, M, dtype=dtype), gap, shift)
            B = Buffer(R, n, dtype, whole(g, 4, R, n, dtype=dtype), gap, shift)
            C = Buffer(G * M, n, F32, whole(g, 8, G * M, n, dtype=F32) if beta else torch.full((G * M, n), NAN), gap,
                       shift)
            ends = ends_of([rows, 0, R - 11 - rows], 6)
            for X in (A, B):
                X.view[:6], X.view[ends[-1]:] = NAN, NAN
            c = matrices(C, G, M, n)
            before = c.clone()
            mp.gemm_grouped_wgrad(A.view.t(), B.view, c, i32(ends), alpha, beta)
            torch.cuda.synchronize()
            for e in range(G):
                here = slice(ends[e], ends[e + 1])
                v = alpha * (A.view[here].double().t() @ B.view[here].double())
                same(c[e], (v + beta * before[e].double() if beta else v).float())
            assert C.outside_untouched()


@pytest.mark.parametrize("kernel", list(ok.WGRAD))
def test_wgrad_wrong_offsets_stay_inside(kernel):
    G, R, M, N = ok.WGRAD[kernel]
    g = generator(G, R, M, N)
    for ends in no_partition(G, R):
        A, B = (Buffer(R, n, BF16, whole(g, 4, R, n, dtype=BF16), 1, 1) for n in (M, N))
        C = Buffer(G * M, N, F32, gap=1, shift=1)
        mp.gemm_grouped_wgrad(A.view.t(), B.view, matrices(C, G, M, N), i32(ends))
        torch.cuda.synchronize()
        assert C.outside_untouched()


# ---- gradients of the rows' way back ----------------------------------------

@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("yt", [F16, BF16, F32])
@pytest.mark.parametrize("gt", [F16, BF16, F32])
@pytest.mark.parametrize("T,k,H", [(9, 5, 119), (7, 3, 256), (7, 3, 265)])
def test_combine_backward_types(dt, yt, gt, T, k, H):
    g = generator(T, k, H)
    R = T * k + 3
    position = torch.randperm(R, generator=g, device=device())[:T * k].int().view(T, k)
    position[2], position[1, 1], position[3, 0] = -1, R, -(1 << 31)
    D = Buffer(T, H, dt, whole(g, 8, T, H, dtype=dt), 1, 1)
    Y = Buffer(R, H, yt, whole(g, 8, R, H, dtype=yt), 3, 0)
    w, dw = powers(g, -2, 2, T, k), torch.full((T, k), NAN, device=device())
    out = Buffer(R, H, gt, gap=2, shift=1)
    mp.combine_rows_backward(D.view, Y.view, position, w, out.view, dw)
    torch.cuda.synchronize()
    want, dots = old(out).clone(), torch.zeros(T, k, device=device())
    for t in range(T):
        for s in range(k):
            p = int(position[t, s])
            if 0 <= p < R:
                want[p] = (w[t, s] * D.view[t].float()).to(gt)
                dots[t, s] = (D.view[t].double() * Y.view[p].double()).sum()
    assert torch.equal(out.view, want) and torch.equal(dw, dots) and out.outside_untouched()
