"""The paged cache (tcq_cache_write, tcq_cache_read) against the definition of its places and
codes: every byte of the cache is compared, those of other tokens included."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import api  # noqa: E402

import mx_check as mc  # noqa: E402
from cache_check import Batch  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]
FORMATS = ["fp4", "fp8"]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _filled(pages, heads, page, dim, fmt):
    c = api.Cache.empty(pages, heads, page, dim, fmt)
    for t in (c.k_codes, c.k_scale, c.v_codes, c.v_scale):
        t.fill_(77)
    return c


def _places(b):
    """(row, page, place) of every new token that is somewhere."""
    out, at = [], 0
    table = b.table.cpu().tolist()
    for s, (n, length) in enumerate(b.sizes):
        for i in range(n):
            p = length - n + i
            if 0 <= p < len(table[s]) * b.page and 0 <= table[s][p // b.page] < b.pages:
                out.append((at + i, table[s][p // b.page], p % b.page))
        at += n
    return out


SIZES = [[(1, 1)], [(1, 5), (1, 64), (1, 33)], [(7, 7), (0, 20), (3, 40), (0, 0), (12, 90)],
         [(100, 300)], [(5, 3), (4, 70)]]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,dim,page", [(1, 64, 1), (2, 64, 16), (8, 128, 32), (3, 256, 64)])
def test_write_and_read(heads, dim, page, dtype, fmt):
    for n, sizes in enumerate(SIZES):
        sys.stdout.write(f"cache {heads}x{dim} page {page} {dtype} {fmt} {sizes}\n")
        sys.stdout.flush()
        g = _gen(n)
        b = Batch(sizes, page, g, extra_rows=2)
        cache = _filled(b.pages, heads, page, dim, fmt)
        want = [t.clone() for t in (cache.k_codes, cache.k_scale, cache.v_codes, cache.v_scale)]
        k = _randn(g, b.rows, heads, dim).to(dtype)
        v = (_randn(g, b.rows, heads, dim) * 3).to(dtype)
        api.cache_write(cache, k, v, *b.where)
        places = _places(b)
        back = [torch.zeros(b.rows, heads, dim, dtype=torch.float64, device="cuda")
                for _ in range(2)]
        if places:
            row, page_of, place = (torch.tensor(t, device="cuda") for t in zip(*places))
            for x, codes, scale, values in ((k, want[0], want[1], back[0]),
                                            (v, want[2], want[3], back[1])):
                c, e = mc.codes_of(x[row], fmt)
                codes[page_of, :, place] = mc.store(c, fmt)
                scale[page_of, :, place] = e
                values[row] = mc.values_of(c, e, fmt)
        for a, w in zip((cache.k_codes, cache.k_scale, cache.v_codes, cache.v_scale), want):
            assert torch.equal(a, w)
        mine = int(b.starts[-1])
        out = [torch.full_like(k, 5.0) for _ in range(2)]
        for t in TYPES:
            rk, rv = api.cache_read(cache, *b.where, b.rows, t,
                                    out=tuple(o.to(t) for o in out))
            assert torch.equal(rk[:mine], back[0][:mine].to(t))
            assert torch.equal(rv[:mine], back[1][:mine].to(t))
            assert bool((rk[mine:] == 5).all()) and bool((rv[mine:] == 5).all())


def test_many_sequences_find_their_rows():
    """More sequences than a search step probes, many of them empty."""
    g = _gen(1)
    for seqs in (63, 64, 65, 130, 4097, 5000):
        new = (torch.rand(seqs, generator=g, device="cuda") < 0.3).long().cpu().tolist()
        b = Batch([(n, n + 2) for n in new], 4, g)
        cache = api.Cache.empty(b.pages, 1, 4, 64)
        k = torch.arange(b.rows, device="cuda").float().view(-1, 1, 1).expand(-1, 1, 64) % 13 + 1
        k = k.contiguous()
        api.cache_write(cache, k, -k, *b.where)
        rk, rv = api.cache_read(cache, *b.where, b.rows, torch.float32)
        assert torch.equal(rk, k) and torch.equal(rv, -k)
        first = [s for s, n in enumerate(new) if n]
        at = b.table[first, 0].long()
        got = mc.values_of(cache.k_codes[at, 0, 2], cache.k_scale[at, 0, 2], "fp8")
        assert torch.equal(got[:, 0], k[:, 0, 0].double())


def test_strides():
    """Keys, values and read-back vectors as slices of one wider tensor."""
    g = _gen(2)
    heads, dim = 4, 64
    b = Batch([(3, 10), (5, 9)], 8, g)
    cache = api.Cache.empty(b.pages, heads, 8, dim, "fp4")
    wide = torch.full((b.rows, 2 * heads + 1, dim + 8), float("nan"), device="cuda")
    k, v = wide[:, 1:1 + heads, 3:3 + dim], wide[:, 1 + heads:, 5:5 + dim]
    k.copy_(_randn(g, b.rows, heads, dim))
    v.copy_(_randn(g, b.rows, heads, dim))
    api.cache_write(cache, k, v, *b.where)
    out = torch.full_like(wide, 9.0)
    rk, rv = out[:, 1:1 + heads, 3:3 + dim], out[:, 1 + heads:, 5:5 + dim]
    api.cache_read(cache, *b.where, b.rows, torch.float32, out=(rk, rv))
    assert torch.equal(rk.double(), mc.quantised(k, "fp4"))
    assert torch.equal(rv.double(), mc.quantised(v, "fp4"))
    rk.fill_(9.0), rv.fill_(9.0)
    assert bool((out == 9).all())


def test_tokens_that_are_nowhere():
    """Pages of -1, past the cache and past the table: not written, read as zeros."""
    g = _gen(3)
    b = Batch([(40, 40)], 8, g)
    b.table[0, 1], b.table[0, 3] = -1, b.pages
    b.lens[0] = 44  # the last four tokens lie behind the table's five pages
    cache = _filled(b.pages, 2, 8, 64, "fp8")
    k = _randn(g, 40, 2, 64)
    api.cache_write(cache, k, k, *b.where)
    touched = (cache.k_scale != 77).any(3).any(1)  # [pages, place]
    assert int(touched.sum()) <= 20
    rk, rv = api.cache_read(cache, *b.where, 40, torch.float32)
    pos = torch.arange(4, 44, device="cuda")
    gone = (pos // 8 == 1) | (pos // 8 == 3) | (pos >= 40)
    want = mc.quantised(k, "fp8")
    want[gone] = 0
    assert torch.equal(rk.double(), want) and torch.equal(rv.double(), want)


def test_nan_marks_its_group():
    g = _gen(4)
    b = Batch([(2, 2)], 4, g)
    cache = api.Cache.empty(b.pages, 1, 4, 64)
    k = _randn(g, 2, 1, 64)
    k[1, 0, 40] = float("inf")
    api.cache_write(cache, k, k, *b.where)
    rk, _ = api.cache_read(cache, *b.where, 2, torch.float32)
    bad = torch.zeros(2, 1, 64, dtype=torch.bool, device="cuda")
    bad[1, 0, 32:] = True
    assert torch.equal(torch.isnan(rk), bad)


def test_cache_past_32_bits():
    """Places past 2^32 bytes of the cache."""
    heads, page, dim = 8, 128, 128
    pages = (1 << 32) // (heads * page * dim) + 8
    cache = api.Cache.empty(pages, heads, page, dim)
    g = _gen(5)
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    k, v = _randn(g, 300, heads, dim), _randn(g, 300, heads, dim)
    api.cache_write(cache, k, v, table, lens, starts)
    rk, rv = api.cache_read(cache, table, lens, starts, 300, torch.float32)
    assert torch.equal(rk.double(), mc.quantised(k, "fp8"))
    assert torch.equal(rv.double(), mc.quantised(v, "fp8"))
    assert int(cache.k_codes[1:pages - 2].max()) == 0
    q = _randn(g, 300, heads, dim).bfloat16()
    o = api.cache_attention(q, cache, table, lens, starts)
    from cache_check import attention
    want, bound = attention(q, rk.double(), rv.double(), 0, dim ** -0.5, torch.bfloat16)
    assert bool(((o.double() - want).abs() <= bound).all())


def test_graph_of_a_decoding_step():
    """Write, attention and read captured once and replayed for changing lengths."""
    g = _gen(6)
    b = Batch([(1, 30), (1, 9)], 16, g)
    cache = api.Cache.empty(b.pages, 2, 16, 64)
    k, v, q = _randn(g, 2, 2, 64), _randn(g, 2, 2, 64), _randn(g, 2, 8, 64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.cache_write(cache, k, v, *b.where)
        o = api.cache_attention(q, cache, *b.where)
        rk, rv = api.cache_read(cache, *b.where, 2, torch.float32)
    for _ in range(4):
        for t in (k, v, q):
            t.copy_(_randn(g, *t.shape))
        b.lens -= 1
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(rk.double(), mc.quantised(k, "fp8"))
        assert torch.equal(rv.double(), mc.quantised(v, "fp8"))
        assert torch.equal(o, api.cache_attention(q, cache, *b.where))
