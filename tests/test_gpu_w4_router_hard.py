"""GPU: the 4-bit and router operators where they can go wrong beside sizes:
infinities and NaN, offsets beyond 32 bits, operands at the end of an
allocation's rows, graphs, streams and threads, wrong index arrays, and the
whole path of a layer of 4-bit experts with its gradient."""
import math
import threading

import pytest
import torch

import dense_mixed_precision_amd as mp
from tests.gpu_util import device
from tests.ops_util import SENTINEL, U32, Buffer, assert_within, offsets_of
from tests.w4_util import BF16, F16, F32, bound, pack, product, random_weights, values

pytestmark = pytest.mark.gpu
SENTINEL.setdefault(torch.uint8, 0xA7)
INF = math.inf
# tokens and channels for each kind of kernel, at K = 160
SHAPES = [(3, 20), (16, 4700), (30, 8100), (61, 9001), (70, 12500), (63, 41001), (130, 24601)]


def weights(N, K, group, dtype, seed=0, *lead):
    g = torch.Generator().manual_seed(seed + N + K)
    _, packed, scale = random_weights(g, N, K, group, dtype, *lead)
    return packed.to(device()), scale.to(device())


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_nonfinite_rows_stay_in_their_rows(M, N, dtype):
    """A row of A with a NaN is NaN, one with an infinity infinite or NaN as its
    products say; a channel with a NaN scale is NaN; nothing else changes."""
    K, group = 160, 32
    g = torch.Generator().manual_seed(M)
    a = torch.randn(M, K, generator=g).to(dtype)
    codes, packed, scale = random_weights(g, N, K, group, dtype)
    codes[:, 5] = torch.where(codes[:, 5] == 0, 1, codes[:, 5])   # every channel takes value 5
    packed = pack(codes)
    clean = torch.empty(M, N, dtype=F32, device=device())
    mp.gemm_w4(a.to(device()), packed.to(device()), scale.to(device()), clean, group=group)
    a[0, 3], a[M - 1, 5] = math.nan, INF
    scale[7, 2] = math.nan
    out = torch.empty_like(clean)
    mp.gemm_w4(a.to(device()), packed.to(device()), scale.to(device()), out, group=group)
    torch.cuda.synchronize()
    assert torch.isnan(out[0]).all() and torch.isnan(out[:, 7]).all()
    keep = [j for j in range(min(N, 40)) if j != 7]
    if M > 1:
        sign = torch.sign(codes[:, 5]).to(device())
        here = torch.arange(N, device=device()) != 7
        assert torch.equal(out[M - 1][here], (sign.float() * INF)[here])
        assert torch.equal(out[1:M - 1][:, keep], clean[1:M - 1][:, keep])


def test_infinite_tokens_times_zero_codes_are_nan():
    a = torch.full((2, 128), INF, dtype=F16, device=device())
    packed = pack(torch.zeros(4, 128, dtype=torch.int64)).to(device())
    out = torch.zeros(2, 4, device=device())
    mp.gemm_w4(a, packed, torch.ones(4, 1, dtype=F16, device=device()), out)
    assert torch.isnan(out).all()


@pytest.mark.parametrize("dtype,big,small", [(F16, 65504.0, 2.0 ** -24), (BF16, 2.0 ** 100, 2.0 ** -130)])
def test_largest_and_smallest_values(dtype, big, small):
    """Largest tokens and scales, and numbers below the normal ones, exactly."""
    K = 128
    codes = torch.zeros(8, K, dtype=torch.int64)
    codes[:, 0], codes[:, 64] = torch.arange(-8, 0), torch.arange(0, 8)
    packed = pack(codes).to(device())
    for a0, s in ((big, 1.0), (small, 1.0), (1.0, small), (big, small)):
        a = torch.zeros(3, K, dtype=dtype, device=device())
        a[0, 0], a[1, 64], a[2, 0] = a0, a0, -a0
        scale = torch.full((8, 1), s, dtype=dtype, device=device())
        out = torch.empty(3, 8, device=device())
        mp.gemm_w4(a, packed, scale, out, group=128)
        want = a.double().cpu() @ (codes.double() * scale.double().cpu()).t()
        got = out.double().cpu()
        # (an FP32 product below the normal numbers keeps half of their step)
        assert ((got - want).abs() <= 2.0 ** -145).all() or torch.equal(got, want)


def test_offsets_beyond_32_bits():
    """The second expert's codes and scales lie past 4 GiB, and so do the last
    rows of tokens and of the result."""
    dev = device()
    N, K, group = 64, 256, 64
    packed, scale = weights(N, K, group, BF16, 1, 2)
    far = (1 << 32) + 128
    Q = torch.zeros(far + N * K // 2, dtype=torch.uint8, device=dev)
    S = torch.zeros(far + N * K // group, dtype=BF16, device=dev)
    Qv = Q.as_strided((2, N, K // 2), (far, K // 2, 1))
    Sv = S.as_strided((2, N, K // group), (far, K // group, 1))
    Qv.copy_(packed)
    Sv.copy_(scale)
    lda = 1 << 22
    rows = 520
    A = torch.zeros((rows - 1) * lda + K, dtype=BF16, device=dev).as_strided((rows, K), (lda, 1))
    C = torch.zeros((rows - 1) * lda + N, dtype=BF16, device=dev).as_strided((rows, N), (lda, 1))
    A.copy_(torch.randn(rows, K, device=dev))
    mp.gemm_w4(A, Qv, Sv, C, group=group, offsets=offsets_of([rows - 9, 9]))
    for here, e in ((slice(0, rows - 9), 0), (slice(rows - 9, rows), 1)):
        exact, mag = product(A[here], packed[e], scale[e], group)
        assert_within(C[here], exact, bound(exact, mag, K, BF16), f"expert {e}")
    del Q, S, A, C
    # quantize and read back rows past 4 GiB
    W = torch.zeros(1039 * (1 << 21) + 96, dtype=F32, device=dev).as_strided((1040, 96), (1 << 21, 1))
    W.copy_(torch.randn(1040, 96, device=dev))
    q, s = torch.empty(1040, 48, dtype=torch.uint8, device=dev), torch.empty(1040, 3, dtype=F16, device=dev)
    mp.quantize_w4(W, q, s, group=32)
    back = torch.empty_like(W.contiguous())
    mp.dequantize_w4(q, s, back, group=32)
    assert float((back - W).abs().max()) <= 0.51 * float(s.float().max())
    assert torch.equal(back.cpu().double(), values(q, s, 96, 32))


@pytest.mark.parametrize("M,N", SHAPES)
def test_same_from_run_to_run_and_captured(M, N):
    """Replays, with other inputs and eager calls between them, give the eager
    call's bits."""
    dev, K = device(), 1000
    packed, scale = weights(N, K, 64, F16)
    a = torch.randn(M, K, device=dev).to(F16)
    out, eager = torch.empty(M, N, dtype=F16, device=dev), torch.empty(M, N, dtype=F16, device=dev)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        mp.gemm_w4(a, packed, scale, out, group=64)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            mp.gemm_w4(a, packed, scale, out, group=64)
    for _ in range(4):
        a.copy_(torch.randn(M, K, device=dev))
        out.fill_(7.0)
        graph.replay()
        mp.gemm_w4(a, packed, scale, eager, group=64)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def router_step(x, ids, w, loss, counts, probs, dx, dw, workspace):
    mp.select_experts(x, ids, w, normalize=False)
    mp.balance_loss(x, ids, loss, counts, probs=probs, workspace=workspace)
    mp.router_backward(x, ids, dx, dweights=dw, normalize=False, counts=counts)


def router_state(T, E, k, seed):
    g = torch.Generator(device=device()).manual_seed(seed)
    dev = device()
    need = mp.mpgemm_balance_workspace(T, E, k)
    return dict(x=torch.randn(T, E, device=dev, generator=g), ids=torch.zeros(T, k, dtype=torch.int32, device=dev),
                w=torch.zeros(T, k, device=dev), loss=torch.zeros(1, device=dev),
                counts=torch.zeros(E + 1, dtype=torch.int32, device=dev), probs=torch.zeros(E, device=dev),
                dx=torch.zeros(T, E, device=dev), dw=torch.randn(T, k, device=dev, generator=g),
                workspace=torch.empty((need + 3) // 4, dtype=torch.int32, device=dev))


@pytest.mark.parametrize("T,E,k", [(7, 5, 2), (3000, 40, 4), (1500, 300, 20)])
def test_router_captured_on_a_dirty_workspace(T, E, k):
    """Two captured steps share a workspace, filled with garbage in between."""
    a, b = router_state(T, E, k, 1), router_state(T, E, k, 2)
    b["workspace"] = a["workspace"]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        router_step(**a)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            router_step(**a)
            router_step(**b)
    for i in range(3):
        for s in (a, b):
            s["x"].copy_(torch.randn(T, E, device=device()))
        a["workspace"].random_(-(1 << 31), (1 << 31) - 1)
        graph.replay()
        torch.cuda.synchronize()
        for s in (a, b):
            c = {n: torch.empty_like(v) if n not in ("x", "dw") else v for n, v in s.items()}
            c["workspace"] = s["workspace"].clone().random_(-5, 5)
            router_step(**c)
            torch.cuda.synchronize()
            for n in ("ids", "w", "loss", "counts", "probs", "dx"):
                assert torch.equal(c[n], s[n]), n


def test_streams_and_threads():
    """Calls of several threads, each on a stream of its own, at once."""
    dev = device()
    jobs = []
    for i in range(4):
        M, N, K = (5, 300, 640) if i % 2 else (150, 2000, 520)
        packed, scale = weights(N, K, 32, BF16, i)
        jobs.append((torch.randn(M, K, device=dev).to(BF16), packed, scale, torch.empty(M, N, device=dev),
                     router_state(500 + i, 64, 4, i), torch.cuda.Stream()))
    torch.cuda.synchronize()
    errors = []

    def work(a, packed, scale, out, state, stream):
        try:
            for _ in range(20):
                mp.gemm_w4(a, packed, scale, out, group=32, stream=stream)
                with torch.cuda.stream(stream):
                    router_step(**state)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not errors
    for a, packed, scale, out, state, _ in jobs:
        again = torch.empty_like(out)
        mp.gemm_w4(a, packed, scale, again, group=32)
        c = {n: torch.empty_like(v) if n not in ("x", "dw") else v for n, v in state.items()}
        router_step(**c)
        torch.cuda.synchronize()
        assert torch.equal(again, out) and all(torch.equal(c[n], state[n]) for n in ("ids", "w", "loss", "counts", "dx"))


def test_wrong_index_arrays_stay_inside_the_operands():
    dev = device()
    packed, scale = weights(40, 200, 64, F16, 0, 3)
    A = Buffer(30, 200, F16, torch.randn(30, 200))
    C = Buffer(30, 40, F32)
    for offsets in ([5, -7, 1 << 30, 3], [-(1 << 31), (1 << 31) - 1, 0, 30], [30, 20, 10, 0], [0, 30, 0, 30]):
        mp.gemm_w4(A.view, packed, scale, C.view, group=64, offsets=torch.tensor(offsets, dtype=torch.int32, device=dev))
        torch.cuda.synchronize()
        assert C.outside_untouched() and A.outside_untouched()
    x = torch.randn(50, 20, device=dev)
    for dtype, bad in ((torch.int32, (1 << 31) - 1), (torch.int64, (1 << 40) + 3), (torch.int64, -(1 << 40))):
        ids = torch.full((50, 3), bad, dtype=dtype, device=dev)
        counts, loss, dx = Buffer(1, 21, torch.int32), Buffer(1, 1, F32), Buffer(50, 20, F32)
        mp.balance_loss(x, ids, loss.view.reshape(1), counts.view.reshape(-1))
        mp.router_backward(x, ids, dx.view, dweights=torch.ones(50, 3, device=dev), counts=counts.view.reshape(-1))
        torch.cuda.synchronize()
        assert counts.view.reshape(-1).tolist() == [0] * 20 + [50] and float(loss.view) == 0.0
        assert torch.equal(dx.view, torch.zeros_like(dx.view))
        assert counts.outside_untouched() and loss.outside_untouched() and dx.outside_untouched()


@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(normalize):
    """Central differences of the framework's own weights and loss.  With step h
    the third derivatives of a softmax times gradients of sum G leave at most
    h^2 * G (each is below 6 * G), and FP32 values of the function, of at most
    G, 64 * u * G / h."""
    dev = device()
    T, E, k, h = 6, 9, 3, 2.0 ** -6
    g = torch.Generator().manual_seed(4)
    x = torch.randn(T, E, generator=g).to(dev)
    dw = torch.randn(T, k, generator=g).to(dev)
    ids, w = torch.empty(T, k, dtype=torch.int32, device=dev), torch.empty(T, k, device=dev)
    mp.select_experts(x, ids, w, normalize=normalize)
    loss, counts = torch.empty(1, device=dev), torch.empty(E + 1, dtype=torch.int32, device=dev)
    mp.balance_loss(x, ids, loss, counts, coefficient=2.0)
    dx = torch.empty_like(x)
    dloss = torch.tensor([3.0], device=dev)
    mp.router_backward(x, ids, dx, dweights=dw, normalize=normalize, counts=counts, dloss=dloss, coefficient=2.0)

    def value(y):
        ids2, w2, l2, c2 = torch.empty_like(ids), torch.empty_like(w), torch.empty_like(loss), torch.empty_like(counts)
        mp.select_experts(y, ids2, w2, normalize=normalize)
        mp.balance_loss(y, ids, l2, c2, coefficient=2.0)
        assert torch.equal(ids2, ids)
        return float((w2.double() * dw.double()).sum() + 3.0 * l2.double())

    total = float(dw.abs().sum()) + 3.0 * 2.0 * E
    for t in range(T):
        for e in range(E):
            up, down = x.clone(), x.clone()
            up[t, e] += h
            down[t, e] -= h
            try:
                diff = (value(up) - value(down)) / (2 * h)
            except AssertionError:
                continue  # another choice of experts: no derivative
            assert abs(diff - float(dx[t, e])) <= (h * h + 64 * U32 / h) * total


@pytest.mark.parametrize("T,E,k,H,F,group", [(33, 8, 2, 200, 96, 32), (400, 16, 4, 512, 256, 128), (1, 4, 2, 128, 64, 64)])
def test_layer_of_4bit_experts(T, E, k, H, F, group):
    """Gate, selection, sort, 4-bit experts, and back to tokens; then the
    gradient of the gate's logits by the weights and the balance loss."""
    dev = device()
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn(T, H, generator=g).to(BF16)
    gate = (torch.randn(E, H, generator=g) / H ** 0.5).to(BF16)
    W = torch.randn(E, F, H, generator=g) / H ** 0.5
    dout = torch.randn(T, F, generator=g)
    X = x.to(dev)
    Q = torch.empty(E, F, (H + 1) // 2, dtype=torch.uint8, device=dev)
    S = torch.empty(E, F, -(-H // group), dtype=BF16, device=dev)
    for e in range(E):
        mp.quantize_w4(W[e].to(dev), Q[e], S[e], group=group)
    logits = torch.empty(T, E, device=dev)
    mp.gemm(X, gate.to(dev).t(), logits)
    ids, w = torch.empty(T, k, dtype=torch.int32, device=dev), torch.empty(T, k, device=dev)
    mp.select_experts(logits, ids, w)
    order, position, offsets = mp.route(ids, E)
    rows = torch.empty(T * k, H, dtype=BF16, device=dev)
    mp.gather_rows(X, order, rows, top_k=k)
    Y = torch.empty(T * k, F, device=dev)
    mp.gemm_w4(rows, Q, S, Y, group=group, offsets=offsets)
    out = torch.empty(T, F, device=dev)
    mp.combine_rows(Y, position, out, weights=w)
    loss, counts = torch.empty(1, device=dev), torch.empty(E + 1, dtype=torch.int32, device=dev)
    mp.balance_loss(logits, ids, loss, counts, coefficient=0.5)
    dY, dw = torch.empty(T * k, F, dtype=BF16, device=dev), torch.empty(T, k, device=dev)
    mp.combine_rows_backward(dout.to(dev), Y, position, w, dY, dw)
    dlogits = torch.empty(T, E, device=dev)
    mp.router_backward(logits, ids, dlogits, dweights=dw, counts=counts, coefficient=0.5)
    torch.cuda.synchronize()

    # the same from the logits on, in 64 bits
    l = logits.cpu().double().requires_grad_()
    chosen = torch.sort(l.detach(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.cpu().long(), chosen)
    wt = torch.softmax(l.gather(1, chosen), 1)
    y = torch.stack([x[t].double() @ values(Q[e], S[e], H, group).t() for t in range(T) for e in chosen[t].tolist()])
    y = y.view(T, k, F)
    o = (wt[..., None] * y).sum(1)
    c = torch.tensor([int((chosen == e).sum()) for e in range(E)]).double()
    aux = 0.5 * E * (c / (T * k) * torch.softmax(l, 1).mean(0)).sum()
    ((o * dout.double()).sum() + aux).backward()
    assert counts.tolist() == c.long().tolist() + [T]
    # products within w4_util's bound of their magnitudes, weights and sums within
    # (2E + 130)u of theirs; the gradient adds F products, k slots and E experts
    mag = torch.stack([x[t].double().abs() @ values(Q[e], S[e], H, group).abs().t()
                       for t in range(T) for e in chosen[t].tolist()]).view(T, k, F)
    err = bound(y, mag, H, F32)
    rel = (2 * E + 130) * U32
    assert_within(out, o.detach(), (wt.detach()[..., None] * (err + 2 * rel * mag)).sum(1), "out")
    assert abs(float(loss) - float(aux.detach())) <= 4 * rel * float(aux.detach())
    ddw = (dout.double().abs()[:, None] * (err + F * U32 * mag)).sum(2).sum(1, keepdim=True)
    top = (dout.double().abs()[:, None] * mag).sum(2).sum(1, keepdim=True) + 0.5 * E
    assert_within(dlogits, l.grad, (2 * ddw + 8 * rel * top).expand(T, E), "dlogits")
