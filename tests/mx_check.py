"""Reference forms of the microscaled operators in float64 (torch, any device), and error bounds
derived from the kernels' arithmetic.

Bounds count roundings as linear_check does: u = 2^-24 for fp32 arithmetic, each of a sum's K
additions allowed a whole fp32 unit (2 u), half(t) relative plus half the subnormals' spacing for
a value stored in type t.
"""
import torch

from linear_check import U, half, tiny

GROUP = 32
TOP = {"fp4": 2, "fp8": 8}
LIMIT = {"fp4": 6.0, "fp8": 448.0}


def table(fmt):
    """The format's non-negative values by code."""
    mantissa, bias, n = (1, 1, 8) if fmt == "fp4" else (3, 7, 127)
    out = []
    for c in range(n):
        e, m = c >> mantissa, (c & ((1 << mantissa) - 1)) / (1 << mantissa)
        out.append(m * 2.0 ** (1 - bias) if e == 0 else (1 + m) * 2.0 ** (e - bias))
    return torch.tensor(out, dtype=torch.float64)


def _power(e):
    """2^e exactly (torch.ldexp takes a float32 power, which the GPU rounds)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def codes_of(x, fmt):
    """(codes uint8 one per value, scale bytes) of x along its last dimension: the nearest value
    by comparing with every one, the even code of two as near."""
    x = x.double()
    pad = -x.shape[-1] % GROUP
    v = torch.nn.functional.pad(x, (0, pad)).unflatten(-1, (-1, GROUP))
    bad = ~torch.isfinite(v).all(-1)
    v = torch.where(bad.unsqueeze(-1), torch.zeros_like(v), v)
    top = v.abs().amax(-1)
    p = torch.frexp(top)[1].int()
    field = torch.where(top < 2.0 ** -126, torch.zeros_like(p), p + 126)
    e = (field - TOP[fmt]).clamp_min(0)
    u = (v.abs() * _power(127 - e).unsqueeze(-1)).clamp_max(LIMIT[fmt])
    t = table(fmt).to(x.device)
    best = torch.zeros_like(u, dtype=torch.long)
    least = (u - t[0]).abs()
    for c in range(1, t.numel()):
        d = (u - t[c]).abs()
        take = (d < least) | ((d == least) & (c % 2 == 0))
        best = torch.where(take, c, best)
        least = torch.minimum(d, least)
    sign = torch.signbit(v) & ~bad.unsqueeze(-1)
    codes = best + sign.long() * (8 if fmt == "fp4" else 128)
    e = torch.where(bad, torch.full_like(e, 255), e)
    return codes.flatten(-2).to(torch.uint8), e.to(torch.uint8)


def store(codes, fmt):
    return codes if fmt == "fp8" else codes[..., 0::2] | (codes[..., 1::2] << 4)


def load(stored, fmt):
    return stored if fmt == "fp8" else torch.stack([stored & 15, stored >> 4], -1).flatten(-2)


def values_of(codes, scale, fmt):
    """float64 values of one code per value and scale bytes."""
    t = table(fmt).to(codes.device)
    sign = 8 if fmt == "fp4" else 128
    m = t[(codes & (sign - 1)).long().clamp_max(t.numel() - 1)]
    v = torch.where(codes >= sign, -m, m).unflatten(-1, (-1, GROUP))
    e = scale.int().unsqueeze(-1)
    p = torch.where(e == 255, torch.full(e.shape, float("nan"), dtype=torch.float64,
                                         device=e.device), _power(e - 127))
    return (v * p).flatten(-2)


def quantised(x, fmt):
    """float64 values that x's codes stand for."""
    return values_of(*codes_of(x, fmt), fmt)[..., :x.shape[-1]]


def gamma(K, t=None):
    """Relative bound of a sum of K exact products (fp32: of bf16 terms, six to a product)."""
    g = 2.0 * (6 * K + 3 if t == torch.float32 else K + 1) * U
    return g / (1.0 - g)


def linear(x, w, bias, residual):
    """(y, sum of term magnitudes) in float64 for values x and w."""
    y = x @ w.t().contiguous()
    mag = x.abs() @ w.abs().t().contiguous()
    if bias is not None:
        y = y + bias.double()
    if residual is not None:
        y = y + residual.double()
    return y, mag


def linear_bound(y, mag, bias, residual, K, t):
    """Elementwise bound on |y_gpu - y|: the sum, one fp32 unit for each of bias and residual, and
    the rounding to t."""
    d = gamma(K) * mag
    for extra in (bias, residual):
        if extra is not None:
            d = d + 2 * U * (y.abs() + extra.double().abs() + d)
    return d + half(t) * (y.abs() + d) + tiny(t)
