"""The 8-bit floating-point linear layers in plain 64-bit arithmetic (torch, any device).

Written from the definition, without the library: groups of 128, power-of-two
scales, e4m3 codes rounded half to even.
"""
import torch

FMAX = 448.0


def exponents(amax):
    """Least e >= -126 with amax <= 448 * 2^e (float64 in, int64 out), by exact comparisons."""
    safe = torch.where(torch.isfinite(amax) & (amax > 0), amax, torch.ones_like(amax))
    e = torch.floor(torch.log2(safe)).to(torch.int64) - 10
    for _ in range(4):  # powers of two and products with them are exact
        e = torch.where(safe > FMAX * torch.exp2(e.double()), e + 1, e)
    e = torch.where(amax > 0, e, torch.full_like(e, -126))
    return torch.clamp(e, min=-126)


def e4m3(u):
    """Nearest e4m3 value (float64 in and out, |u| <= 448), ties to even: 3 mantissa bits, least normal exponent -6."""
    a = torch.clamp(u.abs(), min=2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(a)) - 3)
    return torch.round(u / step) * step


def blocks(v, rows):
    """v [R, C] float64 -> [RB, rows, CB, 128], zeros behind the edges."""
    r, c = v.shape
    rb, cb = -(-r // rows), -(-c // 128)
    out = torch.zeros((rb * rows, cb * 128), dtype=torch.float64, device=v.device)
    out[:r, :c] = v
    return out.view(rb, rows, cb, 128)


def quantise(v, rows):
    """(code values [R', C'] padded to whole groups, scale bytes [RB, CB]) of v [R, C]."""
    t = blocks(v.double(), rows)
    amax = t.abs().amax(3).amax(1)
    bad = ~torch.isfinite(amax)
    e = exponents(amax)
    codes = e4m3(t * torch.exp2(-e.double())[:, None, :, None])
    codes = torch.where(bad[:, None, :, None], torch.full_like(codes, float("nan")), codes)
    byte = torch.where(bad, torch.full_like(e, 255), e + 127)
    return codes.reshape(t.shape[0] * rows, t.shape[2] * 128), byte


def values(codes, byte, rows, r, c):
    """What codes and scale bytes stand for, [r, c]."""
    scale = torch.where(byte == 255, torch.full_like(byte, 0).double() + float("nan"), torch.exp2(byte.double() - 127))
    t = codes.view(byte.shape[0], rows, byte.shape[1], 128) * scale[:, None, :, None]
    return t.reshape(codes.shape)[:r, :c]


def act_values(x):
    return values(*quantise(x, 1), 1, *x.shape)


def weight_values(w):
    return values(*quantise(w, 128), 128, *w.shape)


def silu_mul(h):
    g, u = h.double().chunk(2, dim=1)
    return g / (1 + torch.exp(-g)) * u


def linear(xv, wv, bias=None):
    """(product, sum of magnitudes) of quantised values, both in 64 bits, the bias in both."""
    y, s = xv @ wv.t(), xv.abs() @ wv.abs().t()
    if bias is not None:
        y, s = y + bias.double(), s + bias.double().abs()
    return y, s


def tolerance(y, s, K):
    """How far a bf16 output may be from y.  The sum: products of two e4m3 are exact; one MMA adds 32 of them to the
    accumulator, and aligning the addends to the largest and rounding the result lose at most 2 units of 2^-23
    of what has been added so far (<= s) each step, ceil(K / 32) steps; the bias one more rounding.  The output:
    half a step of bf16 (2^-8 of the value, after the sum's own error)."""
    acc = (-(-K // 32) + 1) * 2.0 ** -22 * s
    return 2.0 ** -8 * (y.abs() + acc) + acc
