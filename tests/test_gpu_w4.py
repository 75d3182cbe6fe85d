"""GPU: 4-bit weights -- rows to codes and back, and products with them --
against their definitions in 64 bits.  Codes, scales and the values read back
are equal to the definition's; bounds of the products are in w4_util.bound."""
import pytest
import torch

import dense_mixed_precision_amd as mp
from tests.gpu_util import device
from tests.ops_util import SENTINEL, Buffer, assert_within, offsets_of
from tests.w4_util import BF16, F16, F32, bound, definition, pack, product, random_weights, values

pytestmark = pytest.mark.gpu
SENTINEL.setdefault(torch.uint8, 0xA7)
TYPES = [F16, BF16, F32]


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(a, b):
    """Equal, NaN at the same places."""
    a, b = a.cpu(), b.cpu()
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a.float()),
                                                                       torch.nan_to_num(b.float()))


def untouched(buf):
    now = buf.flat.clone()
    view = buf.view
    torch.as_strided(now, view.shape, view.stride(), view.storage_offset()).copy_(
        torch.as_strided(buf.before, view.shape, view.stride(), view.storage_offset()))
    return torch.equal(bits(now), bits(buf.before))


def check_pack(w, wt, st, group, gap=0, shift=0):
    N, K = w.shape
    W = Buffer(N, K, wt, w.to(wt), gap, shift)
    Q = Buffer(N, (K + 1) // 2, torch.uint8, gap=gap, shift=shift)
    S = Buffer(N, -(-K // group), st, gap=gap, shift=shift)
    mp.quantize_w4(W.view, Q.view, S.view, group=group)
    torch.cuda.synchronize()
    codes, scale = definition(W.view, st, group)
    assert same(S.view, scale)
    assert torch.equal(Q.view.cpu(), pack(codes))
    assert untouched(Q) and untouched(S)
    for vt in TYPES:
        V = Buffer(N, K, vt, gap=gap, shift=shift)
        mp.dequantize_w4(Q.view, S.view, V.view, group=group)
        torch.cuda.synchronize()
        assert same(V.view, values(Q.view, S.view, K, group).float().to(vt))
        assert untouched(V)


@pytest.mark.parametrize("wt,st", [(a, b) for a in TYPES for b in (F16, BF16)])
@pytest.mark.parametrize("N,K,group,gap,shift", [
    (1, 1, 32, 0, 0), (3, 2, 64, 1, 1), (2, 7, 32, 3, 1), (5, 8, 128, 0, 0), (4, 9, 32, 0, 0), (3, 31, 32, 1, 0),
    (3, 33, 32, 0, 1), (2, 512, 32, 0, 0), (2, 513, 64, 2, 1), (5, 617, 32, 1, 1), (9, 1024, 128, 0, 0),
    (3, 1000, 256, 8, 0), (3, 1300, 512, 0, 1), (2, 3001, 1024, 1, 1), (2, 5000, 1 << 28, 0, 0), (70, 100, 64, 0, 0),
    (0, 64, 32, 0, 0), (4, 0, 32, 0, 0)])
def test_pack_sizes(wt, st, N, K, group, gap, shift):
    g = torch.Generator().manual_seed(N * 7919 + K)
    check_pack(torch.randn(N, K, generator=g) * torch.exp(2 * torch.randn(N, 1, generator=g)), wt, st, group, gap, shift)


@pytest.mark.parametrize("wt,st", [(a, b) for a in TYPES for b in (F16, BF16)])
def test_pack_middles_and_extremes(wt, st):
    info = torch.finfo(wt)
    step = info.tiny * info.eps  # the smallest number
    rows = torch.zeros(14, 128, dtype=torch.float64)
    rows[0] = (torch.arange(128) % 29 - 14) / 2.0           # scale 1: halves are middles
    rows[1] = (torch.arange(128) % 15 - 7) * 0.125
    rows[2, 5], rows[2, 70] = -info.max, info.max / 3
    rows[3] = step * torch.arange(128)                      # below the normal numbers
    rows[4, 0], rows[4, 64] = step, -5 * step
    rows[6, 3], rows[6, 100] = float("inf"), 1.0
    rows[7, 9] = float("nan")
    rows[8, 9], rows[8, 10] = float("-inf"), float("nan")
    rows[9] = info.tiny * (torch.arange(128) - 64)
    rows[10] = -0.0
    rows[11] = torch.linspace(-1, 1, 128) * (info.max / 2)
    rows[12] = torch.finfo(st).tiny * torch.finfo(st).eps * torch.linspace(-20, 20, 128)  # the scale's smallest
    rows[13] = torch.finfo(st).tiny * torch.linspace(-20, 20, 128)
    for group in (32, 64, 128):
        check_pack(rows.float() if wt == F32 else rows, wt, st, group)


def test_pack_next_to_a_middle():
    """FP32 values one step beside the middle of two codes."""
    g = torch.Generator().manual_seed(5)
    top = 7.0 * (torch.rand(64, 1, generator=g) + 1.0)
    scale = (top.double() / 7.0).float().to(F16).double()
    n = torch.randint(-7, 7, (64, 31), generator=g)
    mid = ((n + 0.5) * scale).float()
    way = torch.randint(-1, 2, (64, 31), generator=g)
    x = torch.where(way == 0, mid, torch.nextafter(mid, torch.where(way > 0, torch.inf, -torch.inf)))
    check_pack(torch.cat([x, top], 1), F32, F16, 32)


def check_gemm(M, N, K, group, dtype, out, gap=0, shift=0, bias=False, seed=0):
    g = torch.Generator().manual_seed(M * 31 + N * 7 + K + seed)
    a = torch.randn(M, K, generator=g).to(dtype)
    _, packed, scale = random_weights(g, N, K, group, dtype)
    b = torch.randn(N, generator=g) if bias else None
    A = Buffer(M, K, dtype, a, gap, shift)
    Q = Buffer(N, (K + 1) // 2, torch.uint8, packed, gap, shift)
    S = Buffer(N, -(-K // group), dtype, scale, gap, shift)
    C = Buffer(M, N, out, gap=gap, shift=shift)
    mp.gemm_w4(A.view, Q.view, S.view, C.view, group=group, bias=None if b is None else b.to(device()))
    torch.cuda.synchronize()
    exact, mag = product(a, packed, scale, group, b)
    assert_within(C.view, exact, bound(exact, mag, K, out, b), f"{M}x{N}x{K} group {group} {dtype}")
    assert untouched(C)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group", [32, 64, 128, 256, 1 << 20])
@pytest.mark.parametrize("M,N,K,gap,shift", [
    (1, 1, 1, 0, 0), (1, 1, 2, 0, 0), (2, 3, 7, 1, 1), (1, 33, 8, 0, 0), (3, 5, 31, 1, 0), (4, 40, 32, 0, 0),
    (16, 32, 64, 0, 0), (17, 31, 65, 1, 1), (5, 64, 127, 0, 0), (1, 100, 128, 0, 0), (7, 33, 129, 3, 1),
    (1, 64, 1024, 0, 0), (8, 48, 1025, 0, 1), (33, 70, 257, 8, 0), (16, 16, 2000, 0, 0), (61, 50, 617, 1, 1),
    (3, 20, 0, 0, 0), (64, 33, 4096, 0, 0)])
def test_gemm_few_rows(dtype, group, M, N, K, gap, shift):
    check_gemm(M, N, K, group, dtype, dtype if N % 2 else F32, gap, shift, bias=M % 3 == 1)


# kernel: (rows, columns, K) that take it
KERNELS = {
    "4x16": (3, 70, [128, 129, 260, 1025, 3000]),
    "16x16": (19, 45, [128, 200, 385, 2049]),
    "8x32, 8 waves": (7, 5001, [4096, 4111]),
    "8x32, 4 waves": (5, 4501, [64, 127, 130, 515]),
    "16x32, 8 waves": (16, 4700, [4096, 4230]),
    "16x32, 4 waves": (14, 4801, [100, 131, 640, 777]),
    "32x32": (29, 8190, [77, 128, 270, 513]),
    "64x32": (61, 9001, [96, 128, 391, 905]),
    "64x128": (70, 12500, [128, 135, 257, 650]),
    "64x256": (63, 41001, [128, 129, 384, 523]),
    "128x256": (130, 24601, [128, 264, 391, 777]),
}


def kernel(M, N, K, group, gap=0, groups=0):
    k = mp.mpgemm_w4_query(groups, M, N, K, group, K + gap, (K + 1) // 2 + gap, -(-K // group) + gap)
    name = f"{k['bm']}x{k['bn']}"
    return f"{name}, {k['waves']} waves" if name in ("8x32", "16x32") else name


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group", [32, 64, 128, 512])
@pytest.mark.parametrize("name", list(KERNELS))
def test_gemm_every_kernel(dtype, group, name):
    M, N, depths = KERNELS[name]
    for i, K in enumerate(depths):
        gap, shift = (0, 0) if i % 2 == 0 else (1, 1)
        assert kernel(M, N, K, group, gap) == name
        check_gemm(M, N, K, group, dtype, [F32, dtype, F16 if dtype == BF16 else BF16][i % 3], gap, shift, bias=i == 1)


def check_groups(sizes, behind, N, K, group, dtype, out, gap=0, shift=0, bias=False, start=0):
    """Rows of each group by its own matrix; `behind` rows of none stay."""
    G, M = len(sizes), start + sum(sizes) + behind
    g = torch.Generator().manual_seed(M * 31 + N * 7 + K)
    a = torch.randn(M, K, generator=g).to(dtype)
    _, packed, scale = random_weights(g, N, K, group, dtype, G)
    b = torch.randn(G, N, generator=g) if bias else None
    A = Buffer(M, K, dtype, a, gap, shift)
    Q = Buffer(G * N, (K + 1) // 2, torch.uint8, packed.view(G * N, -1), gap, shift)
    S = Buffer(G * N, -(-K // group), dtype, scale.view(G * N, -1), gap, shift)
    C = Buffer(M, N, out, gap=gap, shift=shift)
    offsets = offsets_of(sizes) + start
    mp.gemm_w4(A.view, Q.view.unflatten(0, (G, N)), S.view.unflatten(0, (G, N)), C.view, group=group,
               bias=None if b is None else b.to(device()), offsets=offsets)
    torch.cuda.synchronize()
    before = torch.as_strided(C.before, C.view.shape, C.view.stride(), C.view.storage_offset())
    at = start
    for e, n in enumerate(sizes):
        here = slice(at, at + n)
        exact, mag = product(a[here], packed[e], scale[e], group, None if b is None else b[e])
        assert_within(C.view[here], exact, bound(exact, mag, K, out, None if b is None else b[e]), f"group {e}")
        at += n
    for rest in (slice(0, start), slice(at, M)):
        assert torch.equal(bits(C.view[rest].contiguous()), bits(before[rest].contiguous()))
    assert untouched(C)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("sizes,behind,N,K,gap,shift,start", [
    ([3, 0, 1, 7], 2, 33, 100, 1, 1, 0), ([0, 0, 0], 4, 40, 64, 0, 0, 0), ([1], 0, 16, 256, 0, 0, 0),
    ([2, 0, 5, 1, 0, 9], 0, 3001, 390, 0, 0, 0), ([17, 40, 0, 3], 5, 2003, 257, 1, 1, 3),
    ([100, 0, 300, 65], 7, 5003, 129, 0, 0, 0), ([200, 1, 0, 290], 1, 9003, 391, 1, 1, 2),
    ([500, 0, 700], 3, 9000, 264, 0, 0, 0), ([70] * 9, 0, 45, 640, 3, 1, 1)])
def test_gemm_groups(dtype, group, sizes, behind, N, K, gap, shift, start):
    check_groups(sizes, behind, N, K, group, dtype, F32 if N % 2 else dtype, gap, shift, bias=N % 4 == 3, start=start)


def test_gemm_many_groups():
    g = torch.Generator().manual_seed(9)
    sizes = torch.randint(0, 4, (200,), generator=g).tolist()
    check_groups(sizes, 3, 100, 300, 64, BF16, BF16)
    check_groups(sizes, 0, 100, 64, 32, F16, F32, gap=1, shift=1)
