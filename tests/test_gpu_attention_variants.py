"""Attention over the paged cache in each of the kernels' forms: NaN groups where a row does not see
every key, batches of more than 64 sequences with large tiles, large pages."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import api  # noqa: E402

import mx_check as mc  # noqa: E402
from cache_check import Batch, attention  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]
FORMATS = ["fp4", "fp8"]
NAN = float("nan")


def _say(msg):
    sys.stdout.write(msg + "\n")
    sys.stdout.flush()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _check(b, heads, group, dim, fmt, dtype, g, k, v, what):
    """Attention over a cache that holds k and v, against float64; places of nobody hold NaN."""
    starts, _ = b.whole()
    cache = api.Cache.empty(b.pages, heads, b.page, dim, fmt)
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(255)
    api.cache_write(cache, k, v, b.table, b.lens, starts)
    kq, vq = mc.quantised(k, fmt), mc.quantised(v, fmt)
    q = _randn(g, b.rows, heads * group, dim).to(dtype)
    o = api.cache_attention(q, cache, *b.where)
    at = key = 0
    for n, length in b.sizes:
        want, bound = attention(q[at:at + n], kq[key:key + length], vq[key:key + length],
                                length - n, dim ** -0.5, dtype)
        got = o[at:at + n].double()
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
        bad = ~nan & ~((got - want).abs() <= bound)
        assert not bool(bad.any()), f"{what}: {int(bad.sum())} outside"
        at, key = at + n, key + length


# few rows, in one run and in several; one tile of rows to a wave and two (bf16, 128 dims, more than
# 256 rows on average), both with runs; both kernels
SIZES = [[(6, 90)], [(3, 5000), (1, 3000)], [(50, 180)], [(150, 400)], [(80, 7000)],
         [(100, 100), (90, 5000)], [(2, 300), (70, 2500), (5, 64)]]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("sizes", SIZES)
def test_nan_reaches_those_who_see_it(sizes, dim, dtype, fmt):
    """A key's or a value's group that stands for NaN, in keys that every query, the later ones or
    only the last one of its sequence sees, and one behind a page's end."""
    _say(f"nan {sizes} {dim} {dtype} {fmt}")
    g = _gen(dim)
    b = Batch(sizes, 16, g)
    _, total = b.whole()
    group = 4
    for which in ("k", "v"):
        for place in ("first", "mid", "last", "page"):
            k, v = _randn(g, total, 2, dim), _randn(g, total, 2, dim)
            key = 0
            for s, (n, length) in enumerate(sizes):
                t = {"first": length - n, "mid": length - 1 - n // 2, "last": length - 1,
                     "page": max(length - n // 3 - 16, 0) // 16 * 16}[place]
                if which == "k":
                    k[key + t, s % 2, 33] = NAN
                else:
                    v[key + t, 1 - s % 2, (37 * s + 32) % dim] = float("inf")
                key += length
            _check(b, 2, group, dim, fmt, dtype, g, k, v, f"{which} {place}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("kind", ["chunks", "both", "tokens"])
def test_more_than_64_sequences(kind, dim, dtype):
    """Items found in the running sums, with tiles of 16, 128 and 256 rows."""
    _say(f"many {kind} {dim} {dtype}")
    g = _gen(7)
    sizes = []
    for s in range(75):
        n = {"chunks": 60 + s * 13 % 70, "both": (1, 90, 7)[s % 3], "tokens": 1 + s % 4}[kind]
        sizes.append((n, n + s * 31 % 200))
    sizes[11] = (sizes[11][0], 4000)
    sizes[70] = (0, 50)
    b = Batch(sizes, 32, g)
    _, total = b.whole()
    k, v = _randn(g, total, 1, dim), _randn(g, total, 1, dim)
    v[3, 0, 5] = NAN
    _check(b, 1, 4, dim, "fp8", dtype, g, k, v, kind)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [512, 4096])
def test_large_pages(page, fmt):
    g = _gen(8)
    for sizes in ([(1, 513), (3, 4100)], [(150, 5000), (1, 20)], [(40, 511)]):
        b = Batch(sizes, page, g)
        _, total = b.whole()
        k, v = _randn(g, total, 2, 128), _randn(g, total, 2, 128)
        _check(b, 2, 4, 128, fmt, torch.bfloat16, g, k, v, f"pages of {page}")
        starts, _ = b.whole()
        cache = api.Cache.empty(b.pages, 2, page, 128, fmt)
        api.cache_write(cache, k, v, b.table, b.lens, starts)
        kr, vr = api.cache_read(cache, b.table, b.lens, starts, total, torch.float32)
        assert torch.equal(kr.double(), mc.quantised(k, fmt))
        assert torch.equal(vr.double(), mc.quantised(v, fmt))
