"""Attention over the paged cache: how the weights of few query rows are held.  16-bit queries'
weights are two bf16 terms, so that what is left of their rounding is far below that of the
output."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import api  # noqa: E402

import mx_check as mc  # noqa: E402
from cache_check import Batch, attention  # noqa: E402
from linear_check import half, tiny  # noqa: E402


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _expect(b, q, k, v, scale):
    """(o, bound) for bf16 queries whose weights are held like those of fp16 ones, to 2^-15: the
    bound of fp16 outputs holds one more rounding than there is, bf16's is added to it."""
    want = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    at = key = 0
    for n, length in b.sizes:
        o, e = attention(q[at:at + n], k[key:key + length], v[key:key + length], length - n, scale,
                         torch.float16)
        want[at:at + n] = o
        bound[at:at + n] = e + half(torch.bfloat16) * (o.abs() + e) + tiny(torch.bfloat16)
        at, key = at + n, key + length
    return want, bound


# single tokens, keys in one run and in several; drafted ones; few rows of a batch that has large
# tiles beside them
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("sizes,few", [([(1, 40), (1, 2), (1, 700)], 3), ([(1, 6000)], 1),
                                       ([(4, 100), (4, 31), (4, 3000)], 3),
                                       ([(3, 90), (2, 2000), (200, 300)], 2)])
def test_few_rows_round_once(sizes, few, dim, fmt):
    sys.stdout.write(f"weights {sizes} {dim} {fmt}\n")
    sys.stdout.flush()
    g = _gen(dim)
    b = Batch(sizes, 16, g)
    starts, total = b.whole()
    cache = api.Cache.empty(b.pages, 2, 16, dim, fmt)
    # (values of both signs: outputs are small beside what the weights' errors multiply)
    k, v = _randn(g, total, 2, dim), _randn(g, total, 2, dim)
    api.cache_write(cache, k, v, b.table, b.lens, starts)
    q = _randn(g, b.rows, 8, dim).bfloat16()
    want, bound = _expect(b, q, mc.quantised(k, fmt), mc.quantised(v, fmt), dim ** -0.5)
    o = api.cache_attention(q, cache, *b.where)
    rows = sum(n for n, _ in sizes[:few])
    off = (o.double() - want).abs()[:rows] / bound[:rows]
    assert float(off.max()) <= 1.0, f"worst {float(off.max()):.3g} of the bound"
