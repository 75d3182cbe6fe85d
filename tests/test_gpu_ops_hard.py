"""GPU: the operator library where calls go wrong most easily: foreign rows
that hold NaN, offsets that do not start at 0, offsets beyond 32 bits, a whole
layer captured and replayed with other experts, several streams and threads at
once, workspaces of the caller's."""
import threading

import pytest
import torch

import dense_mixed_precision_amd as mp
from tests.gpu_util import device
from tests.ops_util import U32, assert_within, order_by_expert

pytestmark = pytest.mark.gpu
NAN = float("nan")


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=device())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("sizes", [[3, 5, 9], [40, 70, 100], [300, 129, 257]])
@pytest.mark.parametrize("col", [False, True])
def test_nan_of_other_rows_and_groups_stays_there(dtype, sizes, col):
    """Rows before the first group, behind the last, and of the middle group
    are NaN; so is the middle group's matrix.  Only the middle group's results
    are NaN, and rows of no group keep what they hold."""
    g = torch.Generator().manual_seed(sum(sizes))
    K, N, first = 77, 150, 6
    ends = [first]
    for n in sizes:
        ends.append(ends[-1] + n)
    R = ends[-1] + 11
    a = torch.randn(R, K, generator=g).to(dtype)
    b = torch.randn(3, N, K, generator=g).to(dtype)
    clean = a.clone()
    a[:first], a[ends[-1]:], a[ends[1]:ends[2]], b[1] = NAN, NAN, NAN, NAN
    out = torch.full((R, N), 7.0, device=device())
    bd = b.to(device())
    mp.gemm_grouped(a.to(device()), bd.mT if col else bd.mT.contiguous(), out, i32(ends))
    dw = torch.empty(3, K, N, device=device())
    y = torch.randn(R, N, generator=g).to(dtype)
    mp.gemm_grouped_wgrad(a.to(device()).t(), y.to(device()), dw, i32(ends))
    torch.cuda.synchronize()
    assert (out[:first] == 7).all() and (out[ends[-1]:] == 7).all()
    assert torch.isnan(out[ends[1]:ends[2]]).all() and torch.isnan(dw[1]).all()
    for e in (0, 2):
        x, w, v = clean[ends[e]:ends[e + 1]].double(), b[e].double(), y[ends[e]:ends[e + 1]].double()
        assert_within(out[ends[e]:ends[e + 1]], x @ w.t(), (K + 2) * U32 * (x.abs() @ w.abs().t()), f"rows of {e}")
        assert_within(dw[e], x.t() @ v, (len(x) + 2) * U32 * (x.abs().t() @ v.abs()), f"weights of {e}")


def test_infinite_values_and_extreme_codes():
    """An infinity in one row of A reaches that row alone; the 8-bit code -128
    is a code like the others."""
    a = torch.ones(70, 64, dtype=torch.float16)
    a[5, 3] = float("inf")
    b = torch.ones(1, 64, 40, dtype=torch.float16, device=device())
    out = torch.empty(70, 40, device=device())
    mp.gemm_grouped(a.to(device()), b, out, i32([0, 70]))
    assert torch.isinf(out[5]).all() and (out[[0, 4, 6, 69]] == 64).all()
    q = torch.full((70, 64), -128, dtype=torch.int8, device=device())
    w = torch.full((40, 64), -128, dtype=torch.int8, device=device())
    one = torch.ones(70, device=device())
    mp.gemm_i8(q, w.t(), out, one, one[:40].contiguous())
    assert (out == 64 * 128 * 128).all()


def test_weights_of_absent_pairs_do_not_count():
    y = torch.randn(4, 50, device=device())
    position = i32([[0, -1], [-1, 3], [-1, -1], [1, 2]])
    w = torch.tensor([[2.0, NAN], [NAN, 0.5], [NAN, float("inf")], [1.0, -1.0]], device=device())
    out = torch.empty(4, 50, device=device())
    mp.combine_rows(y, position, out, weights=w)
    assert torch.equal(out[0], 2 * y[0]) and torch.equal(out[1], 0.5 * y[3]) and (out[2] == 0).all()
    dy, dw = torch.zeros(4, 50, device=device()), torch.empty(4, 2, device=device())
    mp.combine_rows_backward(torch.ones(4, 50, device=device()), y, position, w, dy, dw)
    assert torch.isfinite(dy).all() and torch.isfinite(dw).all()
    assert (dw[2] == 0).all() and dw[0, 1] == 0 and dw[1, 0] == 0


def test_rows_that_are_not_there_may_hold_anything():
    """NaN in rows of Y that no position names, infinities in dropped rows of X."""
    y = torch.full((9, 300), NAN, device=device())
    y[4] = 1.0
    out = torch.empty(2, 300, device=device())
    mp.combine_rows(y, i32([[4, -1, -1, -1, -1], [-1, 4, 4, -1, 4]]), out)
    assert (out[0] == 1).all() and (out[1] == 3).all()


def layer(x, ids, w, slots, order=None):
    T, k = ids.shape
    E, N = w.shape[:2]
    order, position, offsets = mp.route(ids, E)
    rows = torch.zeros(T * k, x.shape[1], dtype=x.dtype, device=x.device)
    y = torch.zeros(T * k, N, device=x.device)
    out = torch.empty(T, N, device=x.device)
    mp.gather_rows(x, order, rows, top_k=k)
    mp.gemm_grouped(rows, w.mT, y, offsets)
    mp.combine_rows(y, position, out, weights=slots)
    return out


def test_layer_captured_and_replayed_with_other_experts():
    """The sizes of the groups are read on the device: a captured layer serves
    every routing of the same number of tokens."""
    g = torch.Generator().manual_seed(1)
    T, k, E, H, N = 150, 3, 9, 128, 200
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(device())
    w = torch.randn(E, N, H, generator=g).to(torch.bfloat16).to(device())
    slots = torch.rand(T, k, generator=g).to(device())
    ids = torch.zeros(T, k, dtype=torch.int32, device=device())
    layer(x, ids, w, slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, ids, w, slots)
    for r in range(4):
        new = torch.randint(-1, E, (T, k), generator=g).to(torch.int32) if r < 3 else torch.full((T, k), -1).int()
        ids.copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, layer(x, ids, w, slots)), f"replay {r}"
    assert (got == 0).all()  # the last one had no experts


def test_two_graphs_share_a_workspace_one_after_the_other():
    T, k, E = 4000, 4, 33
    g = torch.Generator().manual_seed(2)
    ws = torch.empty(mp.mpgemm_route_workspace(T * k, E) // 4, dtype=torch.int32, device=device())
    ids = [torch.randint(0, E, (T, k), generator=g).int().to(device()) for _ in range(2)]
    mp.route(ids[0], E, workspace=ws)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(mp.route(ids[i], E, workspace=ws))
    for _ in range(3):
        for i in (1, 0, 0, 1):
            graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        want = order_by_expert(ids[i].cpu(), E)
        assert outs[i][0].tolist() == want[0] and outs[i][1].reshape(-1).tolist() == want[1]


def test_streams_and_threads_at_once():
    """Eight host threads, each on a stream of its own, with calls that need a
    workspace (allocated per call) and calls that do not."""
    E, T, k = 17, 3000, 3
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, 256, generator=g).to(torch.float16).to(device())
    w = torch.randn(E, 96, 256, generator=g).to(torch.float16).to(device())
    slots = torch.rand(T, k, generator=g).to(device())
    ids = [torch.randint(0, E, (T, k), generator=g).int().to(device()) for _ in range(8)]
    want = [layer(x, i, w, slots) for i in ids]
    torch.cuda.synchronize()
    got, failed = [None] * 8, []

    def work(n):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[n] = layer(x, ids[n], w, slots)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in range(8)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not failed
    for n in range(8):
        assert torch.equal(got[n], want[n])


def test_stream_handles():
    """A raw handle, the default stream's 0, a Stream object."""
    ids = torch.randint(0, 5, (2000, 4), generator=torch.Generator().manual_seed(4)).int().to(device())
    want = order_by_expert(ids.cpu(), 5)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (0, side, side.cuda_stream):
        order, position, offsets = mp.route(ids, 5, stream=s)
        torch.cuda.synchronize()
        assert order.tolist() == want[0] and offsets.tolist() == want[2]


def test_callers_workspaces():
    """Enough, too little and none: the same rows."""
    g = torch.Generator().manual_seed(5)
    T, k, H = 5000, 2, 4096
    x = torch.randn(T, H, generator=g).to(torch.float16).to(device())
    order, _, _ = mp.route(torch.randint(0, 9, (T, k), generator=g).int().to(device()), 9)
    need = mp.mpgemm_rows_workspace(mp.MPGEMM_T_F16, T, H, T * k, k)
    assert need == 4 * T * k
    full = torch.full((need // 4 + 2,), 5, dtype=torch.int32, device=device())
    rows = []
    for ws in (None, full[:need // 4], full[:10]):
        y = torch.zeros(T * k, H, dtype=torch.float16, device=device())
        mp.gather_rows(x, order, y, top_k=k, workspace=ws)
        q, s = torch.zeros(T * k, H, dtype=torch.int8, device=device()), torch.zeros(T * k, device=device())
        mp.quantize_rows(x, q, s, order=order, top_k=k, workspace=ws)
        rows.append((y, q, s))
    torch.cuda.synchronize()
    assert (full[need // 4:] == 5).all()
    for y, q, s in rows[1:]:
        assert torch.equal(y, rows[0][0]) and torch.equal(q, rows[0][1]) and torch.equal(s, rows[0][2])


# ---- offsets beyond 32 bits -------------------------------------------------

def test_more_rows_than_one_dimension_of_a_launch_holds():
    """2^24 + 5 rows: combine takes a workgroup of 256 for each, over 2^32
    threads, the others a wave."""
    dev = device()
    n = (1 << 24) + 5
    x = torch.arange(n, device=dev, dtype=torch.int32).bitwise_and_(127).add_(1).to(torch.float16).view(n, 1)
    q, s = torch.zeros(n, 1, dtype=torch.int8, device=dev), torch.zeros(n, device=dev)
    mp.quantize_rows(x, q, s)
    # (in 64 bits: torch divides FP32 by a number through its reciprocal)
    assert (q == 127).all() and torch.equal(s, (x.double() / 127.0).float().view(-1))
    position = torch.arange(n - 1, -1, -1, device=dev, dtype=torch.int32).view(n, 1)
    out = torch.zeros(n, 1, device=dev)
    mp.combine_rows(x, position, out)
    assert torch.equal(out, x.float().flip(0))
    dy, dw = torch.zeros(n, 1, dtype=torch.float16, device=dev), torch.zeros(n, 1, device=dev)
    mp.combine_rows_backward(out, x, position, None, dy, dw)
    assert torch.equal(dy, x) and torch.equal(dw, out * out)
    y = torch.zeros(n, 1, dtype=torch.float16, device=dev)
    mp.gather_rows(x, position.view(-1), y)
    assert torch.equal(y, x.flip(0))
    ids = torch.arange(n, device=dev, dtype=torch.int32).remainder_(3)
    order, back, offsets = mp.route(ids, 3)
    assert offsets.tolist() == [0, (n + 2) // 3, (n + 2) // 3 + (n + 1) // 3, n]
    at = torch.arange(n, device=dev, dtype=torch.int32)
    assert torch.equal(back[order.long()], at) and torch.equal(ids[order.long()], torch.sort(ids).values)
    assert (order[1:offsets[1]] > order[:offsets[1] - 1]).all()


def test_rows_beyond_32_bits():
    """Rows at more than 2^32 bytes, and 2^31 elements, into each operand."""
    dev = device()
    T, H = 140000, 16384          # 2.3e9 values
    x = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    x.random_(-120, 121)
    x[:, 0] = 127.0
    order = i32([2 * (T - 1), 5, 2 * (T - 3) + 1, -1])
    y = torch.zeros(4, H, dtype=torch.bfloat16, device=dev)
    mp.gather_rows(x, order, y, top_k=2)
    q, s = torch.zeros(T, H, dtype=torch.int8, device=dev), torch.zeros(T, device=dev)
    mp.quantize_rows(x, q, s)
    torch.cuda.synchronize()
    assert torch.equal(y[0], x[T - 1]) and torch.equal(y[1], x[2]) and torch.equal(y[2], x[T - 3]) and (y[3] == 0).all()
    assert (s == 1).all() and torch.equal(q[-3:].float(), x[-3:].float()) and torch.equal(q[:3].float(), x[:3].float())
    out = torch.empty(2, H, device=dev)
    position = i32([[T - 1, 0], [-1, T - 2]])
    mp.combine_rows(x, position, out)
    dy = torch.zeros(T, H, dtype=torch.bfloat16, device=dev)
    dw = torch.empty(2, 2, device=dev)
    mp.combine_rows_backward(out, x, position, None, dy, dw)
    # whole numbers up to 254: exact in FP32
    assert torch.equal(out[0], x[T - 1].float() + x[0].float()) and torch.equal(out[1], x[T - 2].float())
    assert torch.equal(dy[T - 2], out[1].to(torch.bfloat16)) and torch.equal(dy[T - 1], out[0].to(torch.bfloat16))
    assert dw[1, 0] == 0 and (dy[1:T - 2] == 0).all()


def test_products_beyond_32_bits():
    """Weights of the last group, and rows of C, past 2^31 elements and 2^32 bytes."""
    dev = device()
    G, N, K = 70, 8192, 4096       # 2.35e9 weights
    w = torch.zeros(G, N, K, dtype=torch.int8, device=dev)
    w[-1] = 1
    w[-1, -1] = 2
    R = 300000                     # C: 2.46e9 values
    a = torch.ones(R, K, dtype=torch.int8, device=dev)
    c = torch.zeros(R, N, dtype=torch.bfloat16, device=dev)
    ends = [0] * G + [R]
    ends[G - 1] = R - 20
    one = torch.ones(R, device=dev)
    mp.gemm_i8(a, w.mT, c, one, torch.ones(G, N, device=dev), offsets=i32(ends))
    torch.cuda.synchronize()
    assert (c[-20:, :-1] == K).all() and (c[-20:, -1] == 2 * K).all() and (c[:1000] == 0).all()
    assert (c[R - 1000:R - 20] == 0).all()
    del a, c, w
    w = torch.zeros(G, N, K, dtype=torch.bfloat16, device=dev)
    w[-1] = 1
    a = torch.ones(R, K, dtype=torch.bfloat16, device=dev)
    c = torch.full((R, N), 3.0, device=dev)
    mp.gemm_grouped(a, w.mT, c, i32(ends))
    torch.cuda.synchronize()
    assert (c[-20:] == K).all() and (c[:1000] == 0).all()
    dw = torch.full((G, N, K), 3.0, device=dev)
    mp.gemm_grouped_wgrad(c.to(torch.bfloat16).t(), a, dw, i32(ends))
    torch.cuda.synchronize()
    assert (dw[-1] == 20 * K).all() and (dw[0] == 0).all() and (dw[-2] == 0).all()
