"""Attention of many bf16 query rows: weights are fp16 numbers, to 2^-11 of themselves or 2^-32 of the
row's largest, where the values that a workgroup meets are fp16 numbers beside one another, and two
bf16 terms where they are not."""
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

BF16 = torch.bfloat16


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _write(b, k, v, fmt):
    starts, _ = b.whole()
    cache = api.Cache.empty(b.pages, k.shape[1], b.page, k.shape[2], fmt)
    api.cache_write(cache, k, v, b.table, b.lens, starts)
    return cache


def _check(o, b, q, k, v, what):
    """o against float64.  fp16 queries' bound counts everything but two things: the weights' 2^-11
    (twice, for the numerator and the sum, and a sixteenth for second orders, of the weighted mean of
    |v|) and 2^-32 of the largest weight (which is one) for each key, likewise."""
    at = key = 0
    for n, length in b.sizes:
        kk, vv = k[key:key + length], v[key:key + length]
        want, e = attention(q[at:at + n], kk, vv, length - n, q.shape[2] ** -0.5, torch.float16)
        clean = torch.where(torch.isnan(vv), torch.zeros_like(vv), vv).abs()
        size, _ = attention(q[at:at + n], kk, clean, length - n, q.shape[2] ** -0.5, torch.float16)
        all_keys = clean.sum(0).repeat_interleave(q.shape[1] // k.shape[1], 0)[None]
        e = e + (2 + 1 / 16) * (2.0 ** -11 * size + 2.0 ** -32 * (all_keys + length * size))
        bound = e + half(BF16) * (want.abs() + e) + tiny(BF16)
        got = o[at:at + n].double()
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
        off = torch.where(nan, torch.zeros_like(want), (got - want).abs() / bound)
        assert float(off.max()) <= 1.0, f"{what}: {float(off.max()):.3g} of the bound"
        at, key = at + n, key + length


# one tile of rows to a wave and two (128 dims, more than 256 rows on average), in one run and in
# several, beside few rows
SIZES = [[(40, 200)], [(150, 400)], [(100, 6000)], [(70, 70), (1, 90), (300, 2500)]]


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("sizes", SIZES)
def test_weights(sizes, dim, fmt):
    sys.stdout.write(f"weights {sizes} {dim} {fmt}\n")
    sys.stdout.flush()
    g = _gen(dim)
    b = Batch(sizes, 16, g)
    _, total = b.whole()
    k, v = _randn(g, total, 2, dim), _randn(g, total, 2, dim)
    q = _randn(g, b.rows, 8, dim).bfloat16()
    o = api.cache_attention(q, _write(b, k, v, fmt), *b.where)
    _check(o, b, q, mc.quantised(k, fmt), mc.quantised(v, fmt), "weights")


# powers of two by which groups of values differ: key by key, group by group, sequence halves
FAR = {"window": lambda t, c: -15.0 * (t % 2) + 0 * c, "up": lambda t, c: 7.0 * (t > 70) + 0 * c,
       "edges": lambda t, c: torch.where(t < 64, 0.0, (t * 5 + c * 11) % 24 - 16.0),
       "apart": lambda t, c: 40.0 * ((t + c) % 2), "half": lambda t, c: -60.0 + 90.0 * (t > 50),
       "far": lambda t, c: (t * 37 + c * 17) % 161 - 80.0,
       "tiny": lambda t, c: -124.0 + 124.0 * ((t + c) % 3 > 0)}


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("how", list(FAR))
def test_values_far_apart(how, dim, fmt):
    sys.stdout.write(f"far {how} {dim} {fmt}\n")
    sys.stdout.flush()
    g = _gen(3)
    for sizes in ([(90, 150)], [(150, 400), (2, 80)], [(70, 5000), (30, 64)]):
        b = Batch(sizes, 16, g)
        _, total = b.whole()
        t = torch.cat([torch.arange(length, device="cuda") for _, length in sizes])
        c = torch.arange(dim // 32, device="cuda")
        power = FAR[how](t[:, None].float(), c[None, :].float()).expand(total, dim // 32)
        k = _randn(g, total, 2, dim)
        v = _randn(g, total, 2, dim) * torch.exp2(power).repeat_interleave(32, 1)[:, None]
        q = _randn(g, b.rows, 8, dim).bfloat16()
        o = api.cache_attention(q, _write(b, k, v, fmt), *b.where)
        _check(o, b, q, mc.quantised(k, fmt), mc.quantised(v, fmt), how)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_values_of_zero_and_nan(dim, fmt):
    """Groups of zeros, which have the least scale byte, and NaN ones: first, last and between."""
    g = _gen(4)
    for n, length in ((90, 150), (300, 700)):
        for lo, hi, zero in ((0, 70, True), (64, 128, True), (0, length, True), (0, 64, False),
                             (length - 40, length, False)):
            b = Batch([(n, length)], 16, g)
            k, v = _randn(g, length, 2, dim), _randn(g, length, 2, dim)
            v[lo:hi, :, :32] = 0.0 if zero else float("nan")
            v[lo:hi, 1, :] = 0.0
            q = _randn(g, n, 8, dim).bfloat16()
            o = api.cache_attention(q, _write(b, k, v, fmt), *b.where)
            _check(o, b, q, mc.quantised(k, fmt), mc.quantised(v, fmt), f"{lo} {hi} {zero}")


def test_graph_whose_values_change():
    """Replays with values near one another and far apart by turns: nothing of one is left in the next."""
    g = _gen(5)
    sizes, dim = [(150, 400), (3, 60)], 128
    b = Batch(sizes, 16, g)
    starts, total = b.whole()
    cache = api.Cache.empty(b.pages, 2, 16, dim)
    k, v = _randn(g, total, 2, dim), _randn(g, total, 2, dim)
    q = _randn(g, b.rows, 8, dim).bfloat16()
    api.cache_write(cache, k, v, b.table, b.lens, starts)
    api.cache_attention(q, cache, *b.where)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.cache_write(cache, k, v, b.table, b.lens, starts)
        o = api.cache_attention(q, cache, *b.where)
    for far in (False, True, False, True, True, False):
        v.copy_(_randn(g, *v.shape))
        if far:
            v[::3] *= 2.0 ** 50
        graph.replay()
        torch.cuda.synchronize()
        _check(o, b, q, mc.quantised(k, "fp8"), mc.quantised(v, "fp8"), f"far {far}")
        assert torch.equal(o, api.cache_attention(q, cache, *b.where))


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("sizes", [[(90, 200)], [(100, 6000)], [(1, 700), (4, 90)]])
def test_values_of_any_size(sizes, dtype, fmt):
    """Values whose sums, times 2^8 that weights may exceed their reference by, stay below fp32's
    largest number, and values next to its least normal one: outputs scale with them, bit for bit."""
    g = _gen(6)
    b = Batch(sizes, 16, g)
    _, total = b.whole()
    k, v = _randn(g, total, 2, 64), _randn(g, total, 2, 64)
    q = _randn(g, b.rows, 8, 64).to(dtype)
    base = api.cache_attention(q, _write(b, k, v, fmt), *b.where).double()
    top = 125 - 8 - 13
    for power in (top, 60, -60, -100):
        o = api.cache_attention(q, _write(b, k, v * 2.0 ** power, fmt), *b.where).double()
        want = base * 2.0 ** power
        # (outputs near zero are subnormal at the low end; sums of weights times values keep fewer
        # bits only below 2^-126)
        big = want.abs() >= 2.0 ** -112
        assert torch.equal(o[big], want[big]), power
        assert bool(o.isfinite().all())


@pytest.mark.parametrize("fmt,power", [("fp8", 9), ("fp4", 3), ("fp8", -119), ("fp4", -120)])
@pytest.mark.parametrize("dim", [64, 128])
def test_groups_of_zeros_beside_any_size(dim, fmt, power):
    """Groups of zeros (scale byte 0) and of zeros with other bytes, where the first keys' largest
    byte is 128 or next to 0: they stay zeros, and cost no other value a bit."""
    g = _gen(7)
    n, length = 80, 200
    b = Batch([(n, length)], 16, g)
    k, v = _randn(g, length, 2, dim), torch.rand(length, 2, dim, generator=g, device="cuda")
    v = (v + 1.0) * 2.0 ** power * torch.sign(_randn(g, length, 2, dim))
    v[:, :, 32:64] = 0.0
    v[40:60] = 0.0
    q = _randn(g, n, 8, dim).bfloat16()
    cache = _write(b, k, v, fmt)
    o = api.cache_attention(q, cache, *b.where)
    _check(o, b, q, mc.quantised(k, fmt), mc.quantised(v, fmt), f"{power}")
    assert float(o[:, :, 32:64].abs().max()) == 0
    # (groups whose codes are all zero: small values have byte 0 as well)
    zero = (cache.v_codes == 0).unflatten(3, (dim // 32, -1)).all(4)
    assert bool((cache.v_scale[zero] == 0).all())
    for byte in (1, 127, 200, 254):
        cache.v_scale[zero] = byte
        assert torch.equal(api.cache_attention(q, cache, *b.where), o), byte
