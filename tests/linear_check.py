"""Reference forms of the coded linear layer and the 8-bit checkpoints, in float64 (torch,
any device), and error bounds derived from the kernels' arithmetic.

Bounds count roundings: u = 2^-24 for fp32 arithmetic and half(t) = eps(t) / 2 relative
(plus half the spacing of subnormals) for a value stored in type t.  A product's sum of K
terms reaches its result through at most K roundings in any order, each allowed a whole
fp32 unit (2 u), since the matrix instruction's inner sums need not round to nearest:
|sum - exact| <= 2 K u / (1 - 2 K u) * sum |terms|.  fp32 products of
large batches are sums of six exact products of bf16 terms each, which leave out less than
2^-22 = 4 u of the product: 6 K roundings and 4 u more.
"""
import math

import numpy as np
import torch

U = 2.0 ** -24
GROUP = 32


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half the spacing of the type's subnormals."""
    f = torch.finfo(t)
    return f.tiny * f.eps / 2


def gamma(K, t=None):
    """Relative bound of a sum of K products of type t (None: plain fp32 terms)."""
    g = 2.0 * (6 * K + 3 if t == torch.float32 else K + 1) * U
    return g / (1.0 - g)


def random_streams(rng, nb, L, k, V, T):
    nw = (k * T + 31) // 32
    bits = rng.integers(0, 1 << 32, size=(nb, nw), dtype=np.uint64).astype(np.uint32)
    tail = k * T % 32
    if tail:
        bits[:, -1] &= np.uint32(((1 << tail) - 1) << (32 - tail))
    s0 = rng.integers(0, 1 << (L - k * V), size=nb, dtype=np.uint64).astype(np.uint32)
    return bits, s0


def grid_table(L, V, rng):
    """2^L x V multiples of 1/8 up to 4 in magnitude: exact in every layer type."""
    return (rng.integers(-32, 33, size=(1 << L, V)) / 8.0).astype(np.float32)


def act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.where(z <= 0, torch.zeros_like(z), z))
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * torch.sigmoid(-z)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + \
            z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def act_error(z, name):
    """Bound on the fp32 evaluation of act: a few roundings and the library's exp and erf
    (2 units each), relative to |z| (erf's sum with 1 can cancel)."""
    return (0 if name in ("none", "relu") else 8 * 2 * U) * z.abs()


def slope_error(z, name):
    """The same for the slope: terms of size 1 and |z| (|z| phi(z) < 1/4)."""
    return (0 if name in ("none", "relu") else 8 * 2 * U) * (1 + z.abs())


def forward(W, x, a, b, name, res):
    """(z, y) and the bound's parts: sum of term magnitudes for z."""
    s = x @ W.t()
    mag = x.abs() @ W.abs().t()
    z = s if a is None else s * a
    mag = mag if a is None else mag * a.abs()
    if b is not None:
        z = z + b
    y = act(z, name)
    return z, (y if res is None else y + res), mag


def forward_bounds(z, y, mag, res, name, K, t):
    """Elementwise bounds on |z_gpu - z| and |y_gpu - y|."""
    dz = gamma(K, t) * mag + 2 * U * z.abs()
    # |act'| <= 1.13 for silu and gelu, 1 for the others
    dy = 1.13 * dz + act_error(z, name)
    if res is not None:
        dy = dy + 2 * U * (y.abs() + dy)
    return (dz + half(t) * (z.abs() + dz) + tiny(t), dy + half(t) * (y.abs() + dy) + tiny(t))


def pack(x):
    """(codes int8, scale uint8) of the checkpoint's definition, x float64-exact."""
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    v = np.zeros((rows, groups * GROUP))
    v[:, :cols] = x.double().cpu().numpy()
    v = v.reshape(rows, groups, GROUP)
    top = np.where(np.isfinite(v), np.abs(v), np.inf).max(2)
    with np.errstate(divide="ignore", invalid="ignore"):
        _, p = np.frexp(top)
    e = np.where(np.isfinite(top), np.where(top < 2.0 ** -126, 0, p + 126), 255)
    with np.errstate(invalid="ignore", over="ignore"):
        q = np.clip(np.rint(np.ldexp(v, (133 - e)[:, :, None])), -127, 127)
    q = np.where((e == 255)[:, :, None], 0, q)
    return (q.reshape(rows, -1)[:, :cols].astype(np.int8), e.astype(np.uint8))


def unpack(codes, scale):
    """float64 values of a checkpoint (numpy)."""
    cols = codes.shape[1]
    e = np.repeat(scale.astype(np.int64), GROUP, axis=1)[:, :cols]
    v = np.ldexp(codes.astype(np.float64), e - 133)
    return np.where(e == 255, np.nan, v)
