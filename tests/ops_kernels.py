"""For every kernel that a product of the operator library can take, sizes
that take it (checked on the CPU by test_ops_query_host, and by the GPU tests
before they run)."""
import dense_mixed_precision_amd as mp

ROW, COL = mp.MPGEMM_ROW_MAJOR, mp.MPGEMM_COL_MAJOR
# K around the 16-byte vectors and the tiles of 128 and 256 codes, the second
# list for kernels that only long K takes
I8_TAILS = [0, 1, 15, 16, 17, 31, 64, 127, 128, 129, 143, 256, 271, 509]
I8_LONG = [513, 520, 527, 528, 640, 769, 1031]
# K around the vectors of 8 values and the tiles of 64 and 128
TAILS = [0, 1, 7, 8, 9, 31, 63, 64, 65, 72, 127, 130, 200, 255]
MIDDLE = [257, 264, 300, 391]
LONG = [513, 520, 577, 583, 640]

# kernel: (rows, columns, K)
I8 = {
    "narrow, 8 waves": (3, 20, I8_TAILS + I8_LONG),
    "narrow, 4 waves": (16, 16401, I8_TAILS + I8_LONG),
    "16x64x256, 4 stages": (40, 2801, I8_TAILS + I8_LONG),
    "64x64x256, 3 stages": (40, 8201, I8_TAILS + I8_LONG),
    "64x128x128, 3 stages": (40, 16501, I8_TAILS + I8_LONG),
    "128x128x128, 2 stages": (70, 24601, I8_TAILS),
    "128x128x128, 3 stages": (70, 24601, I8_LONG),
    "128x256x128, 3 stages": (70, 32901, I8_LONG),
    "256x256x128, 2 stages": (140, 32901, I8_TAILS + I8_LONG),
}
# kernel: (groups, rows, columns, K)
I8_GROUPS = {
    "narrow, 8 waves": (5, 50, 37, [0, 100, 271]),
    "narrow, 4 waves": (5, 60, 8201, [0, 100, 271]),
    "16x64x256, 4 stages": (5, 120, 2801, [0, 15, 271, 1031]),
    "64x64x256, 3 stages": (2, 100, 2801, [0, 15, 271, 1031]),
    "64x128x128, 3 stages": (5, 300, 2801, [0, 15, 271, 513]),
    "128x128x128, 2 stages": (5, 600, 4101, [0, 15, 271]),
    "128x128x128, 3 stages": (5, 600, 4101, [513, 640]),
    "128x256x128, 3 stages": (5, 1000, 3301, [513, 640]),
    "256x256x128, 2 stages": (4, 700, 8301, [0, 15, 271, 513]),
}
# (kernel, storage order of B): (groups, rows, columns, K)
GROUPED = {
    ("narrow, 8 waves", COL): (5, 50, 37, TAILS + MIDDLE + LONG),
    ("narrow, 4 waves", COL): (5, 60, 2801, TAILS + MIDDLE),
    ("32x64x128, 3 stages", COL): (5, 300, 2801, TAILS + MIDDLE + LONG),
    ("32x64x128, 3 stages", ROW): (5, 50, 37, TAILS + MIDDLE + LONG),
    **{(k, lb): case for lb in (ROW, COL) for k, case in {
        "64x128x64, 3 stages": (5, 200, 8201, TAILS + MIDDLE),
        "128x128x64, 2 stages": (5, 600, 4101, TAILS),
        "128x128x64, 3 stages": (5, 600, 4101, MIDDLE + LONG),
        "128x256x64, 3 stages": (5, 1000, 3301, LONG),
        "256x256x64, 2 stages": (4, 700, 8301, TAILS + LONG),
    }.items()},
}
# kernel: (groups, rows, rows and columns of C)
WGRAD = {
    "64x64x64, 2 stages": (3, 300, 70, 90),
    "128x128x64, 2 stages": (3, 300, 700, 1101),
    "128x256x64, 3 stages": (3, 1600, 900, 2101),
    "256x256x64, 2 stages": (3, 400, 1500, 2001),
}


def name(kernel):
    """A query's answer as the tables above call it."""
    if kernel["narrow"]:
        return f"narrow, {kernel['waves']} waves"
    return f"{kernel['bm']}x{kernel['bn']}x{kernel['bk']}, {kernel['stages']} stages"


def i8_kernel(groups, M, N, K, gap=0):
    ld = max(K + gap, 1)
    return name(mp.mpgemm_i8_query(groups, M, N, K, ld, ld))


def grouped_kernel(layout_b, groups, R, N, K, gap=0):
    return name(mp.mpgemm_grouped_query(layout_b, groups, R, N, K, max(K + gap, 1),
                                        max((N if layout_b == ROW else K) + gap, 1), N + gap))


def wgrad_kernel(groups, R, M, N, gap=0):
    return name(mp.mpgemm_grouped_wgrad_query(groups, R, M, N, M + gap, N + gap, N + gap))
