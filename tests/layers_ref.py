"""64-bit references of the norm with the residual's addition and of the 4-bit products, with bounds of
what the library may be off by (CPU tensors in, float64 out).

How the bounds are made: an output of 16 or 8 bits is rounded once, by at most half a step; everything
before it is in 32 bits.  A matrix instruction's result is taken as off by at most 2^-22 of the sum of its
terms' magnitudes (32 products and the running sum; twice a 32-bit step for the alignment of its terms).
The scaled instruction for 8-bit rows cuts products: of eight neighbouring inputs, each to a multiple of 2^-13 of
the largest one's power of two, towards zero."""
import math

import torch

E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
BF, FH, F8, E8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.float8_e8m0fnu


def half_step(y, dtype):
    """Half a step of dtype at y: relative, or of its smallest numbers."""
    low = {BF: 2.0 ** -134, FH: 2.0 ** -25, F8: 2.0 ** -10, torch.float32: 2.0 ** -150}[dtype]
    return (y.abs() * (torch.finfo(dtype).eps / 2)).clamp(min=low)


def powers(scale):
    e = scale.view(torch.uint8).to(torch.int64)
    return torch.where(e == 255, math.nan, torch.ldexp(torch.ones(()).double(), e - 127))


# ------------------------------------------------------------------------------------- norm

def norm(x, weight, residual, eps):
    """(y, h): y is off by at most 2^-18 |y| in 32 bits: a thread adds up to 32 squares, ten more steps
    join the threads, so mean(h^2) is off by at most 2^-18 of itself, its root by half of that; the
    square root, two divisions and two products add 2^-21."""
    h = x.double() if residual is None else x.double() + residual.double()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    return y if weight is None else y * weight.double(), h


NORM_REL = 2.0 ** -18


# ------------------------------------------------------------------------------------- products

def weights(codes, scales, fmt, group):
    """(w [n][k], magnitude that enters the matrix cores [n][k], scale of each input [n][k])"""
    k = 2 * codes.shape[1]
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(1).long()
    if fmt == "mx":
        v, s = E2M1[c], powers(scales)
        mag = v.abs()
    else:
        v, s = torch.where(c > 7, c - 16, c).double(), scales.double()
        mag = v + 24 + 24  # code + 24, and 24 once more for the sum that takes it back
    s = s.repeat_interleave(group, 1)[:, :k]
    return v * s, mag * s.abs(), s


def rows_of(x, x_scale):
    x = x.double()
    return x if x_scale is None else x * powers(x_scale).repeat_interleave(32, -1)


def product(x, x_scale, codes, scales, fmt, group):
    """(y, bound before the output's rounding).  A chain holds at most eight instructions per group of
    128 (INT), and one per 32 or 128 inputs otherwise, whose running sums are bounded by the whole sum of
    magnitudes; the sums of groups and of waves add K / 32 + 16 roundings of 2^-24."""
    w, mag, _ = weights(codes, scales, fmt, group)
    x = rows_of(x, x_scale)
    k = w.shape[1]
    y = x @ w.t()
    per = 8 if fmt == "int" else 1
    tops = x.abs() @ mag.t()
    plain = x.abs() @ w.abs().t()
    # instructions see the sums of their own group (INT); an MX chain runs through the whole row, its
    # roundings of the running sum add up like k / 32 steps of a sum that grows to `plain`
    chain = per * 2.0 ** -22 * tops if fmt == "int" else (k / 32 + 1) * 2.0 ** -24 * plain + 2.0 ** -22 * plain
    if x_scale is not None:  # seven of eight products cut by less than 2^-13 of the eighth
        top_x = x.abs().unflatten(1, (-1, 8)).amax(-1)
        top_w = w.abs().unflatten(1, (-1, 8)).amax(-1)
        chain = chain + 7 * 2.0 ** -13 * (top_x @ top_w.t())
    return y, chain + (k / 32 + 16) * 2.0 ** -24 * plain


def linear(x, x_scale, codes, scales, fmt, group, bias, dtype):
    y, b = product(x, x_scale, codes, scales, fmt, group)
    if bias is not None:
        y = y + bias.double()
        b = b + 2.0 ** -24 * (y.abs() + bias.double().abs())
    return y, b * (1 + 2.0 ** -8) + half_step(y, dtype)


ACT = {"silu": lambda a: a * torch.sigmoid(a),
       "gelu": lambda a: a * torch.special.ndtr(a),
       "gelu_tanh": lambda a: 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))}


def gated(x, x_scale, gate, up, fmt, group, act, dtype):
    """The activations' slopes stay below 1.13 in size; exp, erf and tanh in 32 bits are taken as off by 2^-20 of
    the activation's argument."""
    a, ba = product(x, x_scale, *gate, fmt, group)
    u, bu = product(x, x_scale, *up, fmt, group)
    f = ACT[act](a)
    y = f * u
    df = 1.13 * ba + 2.0 ** -20 * a.abs()
    b = df * (u.abs() + bu) + f.abs() * bu + 2.0 ** -22 * y.abs()
    return y, b * (1 + 2.0 ** -8) + half_step(y, dtype)


# ------------------------------------------------------------------------------------- inputs

def make_weight(n, k, fmt, group, g, scale_dtype=BF, spread=0):
    """Codes and scales of a layer: every code occurs; MX scales over 2^-spread .. 1."""
    codes = torch.randint(0, 256, (n, k // 2), generator=g).to(torch.uint8)
    groups = -(-k // group)
    if fmt == "mx":
        e = 127 - 3 - torch.randint(0, spread + 1, (n, groups), generator=g)
        return codes, e.to(torch.uint8).view(E8)
    return codes, (0.005 + 0.02 * torch.rand((n, groups), generator=g)).to(scale_dtype)


def make_rows(rows, k, dtype, g):
    """(x, x_scale)"""
    x = torch.randn((rows, k), generator=g)
    if dtype != F8:
        return x.to(dtype), None
    e = torch.randint(114, 126, (rows, k // 32), generator=g).to(torch.uint8)
    return (x * 40).to(F8), e.view(E8)
