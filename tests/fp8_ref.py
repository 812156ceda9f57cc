"""8-bit operands in 64 bits, from their description: packing, values and
the order of the exponents.  Shared by the tests of the 8-bit products."""
import math

import torch

D = torch.float64
HALF_BF16, HALF_E4M3 = 2.0 ** -8, 2.0 ** -4  # half a step, relative to the value


def two_to(k):
    """2^k by its bits: pow(2, k) may be off in the last one, and halves would then round the other way."""
    return ((k.to(torch.int64) + 1023) << 52).view(D)


def exponents(top):
    """k of the smallest power of two, at least 2^-127, whose 448-fold reaches top (float64)."""
    m, x = torch.frexp(top)
    k = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(top == 0, torch.full_like(k, -127), k).clamp(min=-127).to(torch.int64)


def round_e4m3(t):
    """t (|t| <= 448) on e4m3's grid, to nearest even: 3 bits after the first, steps of 2^-9 below 2^-6."""
    _, x = torch.frexp(t)
    step = two_to((x.to(torch.int64) - 1).clamp(min=-6) - 3)
    return torch.round(t / step) * step


def pack(x, tiles=False):
    """(values, k) of x [R, C]: the values that the operand stands for, float64 [R, C], and its exponents [R, ceil(C/128)]."""
    x = x.to(D)
    R, C = x.shape
    u = torch.zeros((R, -(-C // 128) * 128), dtype=D, device=x.device)
    u[:, :C] = x
    b = u.view(R, -1, 128)
    top = torch.where(torch.isfinite(b), b.abs(), torch.zeros_like(b)).amax(2)
    if tiles:
        for r in range(0, R, 128):
            top[r:r + 128] = top[r:r + 128].amax(0, keepdim=True)
    k = exponents(top)
    t = b / two_to(k)[..., None]
    v = torch.where(torch.isfinite(b), round_e4m3(torch.where(torch.isfinite(b), t, torch.zeros_like(t))), torch.full_like(t, math.nan))
    return (v * two_to(k)[..., None]).view(R, -1)[:, :C], k


def exponents_of(e, R, B):
    """k [R, B] of an operand's exponents, element by element."""
    r, b = torch.arange(R, device=e.device)[:, None], torch.arange(B, device=e.device)[None, :]
    return e[r // 128, b // 4, r % 32 * 16 + r % 128 // 32 * 4 + b % 4].to(torch.int64) - 127


def values(op, C):
    """The values [R, C] that an operand (q, e) stands for."""
    q, e = op
    R, P = q.shape
    k = exponents_of(e, R, P // 128)
    return (q.to(torch.float32).to(D).view(R, -1, 128) * two_to(k)[..., None]).view(R, P)[:, :C]


def gelu(h):
    return h * torch.special.erfc(-h / math.sqrt(2)) / 2


def gelu_prime(h):
    return torch.special.erfc(-h / math.sqrt(2)) / 2 + h * torch.exp(-h * h / 2) / math.sqrt(2 * math.pi)


def sum_error(a, b):
    """A bound on the error of a b^T summed in fp32 in any order, products exact: each of the K additions is off by at most
    one unit in the last place (2^-23, for a sum that is cut off) of a partial sum, at most sum |a b|."""
    return (a.shape[1] + 8) * 2.0 ** -23 * (a.abs() @ b.abs().t())


def assert_within(got, want, slack, what=""):
    """|got - want| <= half a bf16 step of the value and `slack`, everywhere."""
    got = got.to(D)
    over = (got - want).abs() - (HALF_BF16 * want.abs() + (1 + HALF_BF16) * slack + 2.0 ** -133)
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    assert float(over.max()) <= 0, f"{what}: over its bound by {float(over.max()):.3e} at a value of {float(want.flatten()[over.argmax()]):.3e}"
