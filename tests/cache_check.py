"""Batches for the paged cache and reference attention in float64, with a bound on what the
kernels' arithmetic may be off by.

A score is off by gamma(D) of its terms' magnitudes, and by 16 fp32 roundings of the largest on
its way through the factor, the running maximum and the exponential's argument; a weight by that
in its exponent and 2^-21 of the exponential itself.  Weights meet the values rounded to their
terms: one bf16 number has 8 bits, so half a step is 2^-8 of it; the first of two is cut off below
2^-7 and the second rounds that by 2^-8 of it, 2^-15; three hold every bit of an fp32 number.  The
weights' sum is that of the rounded ones: with errors of at most r in each, o = N / S is off by at
most r sum p|v| / sum p from N and r |o| from S, each no more than r of the same size, and by second
orders below r / 16 of it.  Sums over keys take one whole fp32 unit per
key and eight per tile of 32 keys (rescaling).  Numerator and denominator count alike.
"""
import math

import torch

import mx_check as mc
from linear_check import U, half, tiny

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -15, torch.float32: 0.0}


class Batch:
    """Sequences of given (new, length), pages of `page` tokens in a shuffled order."""

    def __init__(self, sizes, page, g, spare=3, extra_rows=0, device="cuda"):
        self.sizes, self.page = sizes, page
        need = [-(-max(length, 0) // page) for _, length in sizes]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g, device=device).int()
        self.table = torch.full((len(sizes), max(need + [1])), -1, dtype=torch.int32,
                                device=device)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.free = order[at:]
        new = [n for n, _ in sizes]
        self.lens = torch.tensor([length for _, length in sizes], dtype=torch.int32, device=device)
        self.starts = torch.tensor([sum(new[:s]) for s in range(len(sizes) + 1)],
                                   dtype=torch.int32, device=device)
        self.rows = sum(new) + extra_rows

    @property
    def where(self):
        return self.table, self.lens, self.starts

    def whole(self):
        """starts and rows that make every token of every sequence a new one."""
        lens = [max(length, 0) for _, length in self.sizes]
        return torch.tensor([sum(lens[:s]) for s in range(len(lens) + 1)], dtype=torch.int32,
                            device=self.lens.device), sum(lens)


def attention(q, k, v, first, scale, dtype, there=None):
    """(o, bound) in float64 for one sequence: q [n, Hq, D] at positions first .. first + n - 1, k
    and v [length, H, D] (values that the cache stands for); there: keys that can be seen."""
    n, Hq, D = q.shape
    length, H, _ = k.shape
    out = torch.zeros(n, Hq, D, dtype=torch.float64, device=q.device)
    bound = torch.full_like(out, tiny(dtype))
    if length == 0 or n == 0:
        return out, bound
    pos = torch.arange(first, first + n, device=q.device)
    sees = torch.arange(length, device=q.device)[None, :] <= pos[:, None]
    if there is not None:
        sees = sees & there[None, :]
    some = sees.any(1)
    for h in range(Hq):
        kh, vh = k[:, h * H // Hq], v[:, h * H // Hq]
        x = q[:, h].double()
        s = (x @ kh.t().contiguous()) * scale
        mag = (x.abs() @ kh.abs().t().contiguous()) * scale
        # what a query does not see reaches it in no way
        s = torch.where(sees, s, torch.full_like(s, -math.inf))
        top = torch.where(sees, mag, torch.zeros_like(mag)).amax(1, keepdim=True)
        p = torch.exp(s - s.amax(1, keepdim=True))
        p = torch.where(some[:, None], p, torch.zeros_like(p))
        total = p.sum(1, keepdim=True)
        total = torch.where(some[:, None], total, torch.ones_like(total))
        clean = torch.isfinite(vh).all(1)
        vv = torch.where(torch.isfinite(vh), vh, torch.zeros_like(vh))
        o = p @ vv / total
        if not bool(clean.all()):
            bad = (~torch.isfinite(vh)).double()
            o = torch.where(sees.double() @ bad > 0, torch.full_like(o, math.nan), o)
        size = p @ vv.abs() / total
        ds = (mc.gamma(D) + 16 * U) * top
        e = 2 * (torch.expm1(ds) + 2.0 ** -21) + (2 + 1 / 16) * ROUND[dtype] + \
            4 * U * (length + 8 * (length // 32 + 4))
        out[:, h] = o
        bound[:, h] = e * size + half(dtype) * (o.abs() + e * size) + tiny(dtype)
    return out, bound
