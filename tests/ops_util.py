"""Helpers of the operator tests: device tensors inside sentinel margins, an
order of pairs by expert computed plainly, and error bounds."""
import torch

from tests.gpu_util import device

SENTINEL = {torch.int8: 99, torch.int32: -777, torch.float32: -12345.5, torch.float16: -1234.5,
            torch.bfloat16: -1232.0}
U32 = 2.0 ** -24                 # half a step of FP32
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# half of the smallest step (fixed below the smallest normal number)
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


class Buffer:
    """A rows x cols device view with leading dimension cols + gap, `shift`
    elements off an aligned base, sentinels everywhere else."""

    def __init__(self, rows, cols, dtype, values=None, gap=0, shift=0):
        ld = max(cols + gap, 1)
        span = (rows - 1) * ld + cols if rows and cols else 0
        self.flat = torch.full((64 + shift + span + 64,), SENTINEL[dtype], dtype=dtype, device=device())
        self.view = torch.as_strided(self.flat, (rows, cols), (ld, 1), 64 + shift)
        if values is not None:
            self.view.copy_(values)
        self.before = self.flat.clone()

    def outside_untouched(self):
        """Everything but the view is as it was."""
        now = self.flat.clone()
        torch.as_strided(now, self.view.shape, self.view.stride(), self.view.storage_offset()).copy_(
            torch.as_strided(self.before, self.view.shape, self.view.stride(), self.view.storage_offset()))
        bits = {1: torch.int8, 2: torch.int16, 4: torch.int32}[now.element_size()]
        return torch.equal(now.view(bits), self.before.view(bits))


def order_by_expert(ids, E):
    """(order, position, offsets) as lists, by definition."""
    flat = ids.reshape(-1).tolist()
    order, offsets = [], [0]
    rows = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            rows[e].append(i)
    for e in range(E):
        order += rows[e]
        offsets.append(len(order))
    position = [-1] * len(flat)
    for p, i in enumerate(order):
        position[i] = p
    return order + [-1] * (len(flat) - len(order)), position, offsets


def offsets_of(sizes):
    out = [0]
    for n in sizes:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=device())


def assert_within(got, exact, bound, what):
    """|got - exact| <= bound elementwise, both finite (exact in 64 bits)."""
    got = got.double().cpu()
    exact, bound = exact.cpu(), bound.cpu()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    excess = (got - exact).abs() - bound
    worst = int(excess.argmax()) if excess.numel() else 0
    assert excess.numel() == 0 or float(excess.max()) <= 0, (
        f"{what}: element {worst}: got {got.reshape(-1)[worst]}, exact {exact.reshape(-1)[worst]}, "
        f"bound {bound.reshape(-1)[worst]}")
