"""Helpers of the 4-bit tests: codes and bytes, the definitions in 64 bits, and
error bounds."""
import torch

from tests.ops_util import HALF_STEP, TINY, U32

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def pack(codes):
    """Bytes of N x K codes (-8 .. 7), low nibble first; the spare nibble is 8."""
    q = (codes.to(torch.int64) + 8).cpu()
    if q.shape[-1] % 2:
        q = torch.cat([q, torch.full_like(q[..., :1], 8)], -1)
    return (q[..., 0::2] + 16 * q[..., 1::2]).to(torch.uint8)


def unpack(packed, K):
    """N x K codes of bytes."""
    q = packed.cpu().to(torch.int64)
    return torch.stack([q % 16, q // 16], -1).flatten(-2)[..., :K] - 8


def values(packed, scale, K, group):
    """What codes and scales stand for, in 64 bits (exact)."""
    s = scale.cpu().double().repeat_interleave(group, -1)[..., :K]
    return unpack(packed, K).double() * s


def definition(w, dtype, group):
    """(codes, scale of `dtype`) by definition, on the CPU: m / 7 rounded to FP32
    (64 bits first: a quotient of 24-bit numbers whose 53-bit rounding lies in
    the middle of two FP32 numbers lies there itself) and to dtype; quotients
    value / scale in 64 bits (24 by 11 bits: none is nearer than 2^-37 to a
    middle without being one)."""
    w = w.cpu()
    N, K = w.shape
    groups = -(-K // group)
    x = torch.zeros(N, groups * group, dtype=torch.float64)
    x[:, :K] = w.double()
    x = x.view(N, groups, group)
    bad = ~torch.isfinite(x).all(2)
    top = torch.where(bad, 0.0, x.abs().amax(2)) if K else x.new_zeros(N, 0)
    scale = (top / 7.0).float().to(dtype)
    bad |= ~torch.isfinite(scale)
    scale = torch.where(bad, torch.full_like(scale, float("nan")), scale)
    live = ~bad & (scale > 0)
    step = torch.where(live, scale.double(), 1.0)[..., None]
    codes = torch.where(live[..., None], torch.round(x / step).clamp(-8, 7), 0.0)
    return codes.view(N, groups * group)[:, :K].to(torch.int64), scale


def product(a, packed, scale, group, bias=None):
    """(A @ W.T + bias, sum of magnitudes) in 64 bits, on the CPU."""
    K = a.shape[1]
    w, x = values(packed, scale, K, group), a.cpu().double()
    out, mag = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        out = out + bias.cpu().double()
    return out, mag


def bound(exact, mag, K, dtype, bias=None):
    """How far a product may be from the exact one.  A code times a 16-bit value
    is exact in FP32.  At most 128 products make a chain of FP32 sums, each off
    by at most one step (2u: whether the matrix instruction rounds or cuts); a
    chain's product with its scale joins the sum of the others by one rounding
    (u), K/32 of them at most; 8 waves' sums are 8 more, the bias one.  Each is
    relative to what has been summed, at most `mag` (plus the bias).  Then half a
    step of the output type."""
    steps = 2 * min(K, 128) + -(-K // 32) + 10
    top = mag if bias is None else mag + bias.cpu().double().abs()
    err = 1.01 * steps * U32 * top + 2.0 ** -140
    return err + HALF_STEP[dtype] * (exact.abs() + err) + TINY[dtype]


def random_weights(g, N, K, group, dtype, *lead):
    """(codes, bytes, scale) of normal weights with a scale per group."""
    codes = (2.4 * torch.randn(*lead, N, K, generator=g)).round().clamp(-8, 7).to(torch.int64)
    scale = (0.05 * torch.exp(0.5 * torch.randn(*lead, N, -(-K // group), generator=g))).to(dtype)
    return codes, pack(codes), scale
