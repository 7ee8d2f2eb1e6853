"""Attention over the paged cache (tcq_cache_attention) against a plain form in float64, within a
bound counted from the kernels' roundings (cache_check), and exactly where every weight is one."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import _lib, api  # noqa: E402

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


def _fill(b, heads, dim, fmt, g, k=None, v=None):
    """A cache that holds whole sequences, and the values it stands for."""
    starts, total = b.whole()
    cache = api.Cache.empty(b.pages, heads, b.page, dim, fmt)
    # what belongs to nobody would show
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(0x7E if fmt == "fp8" else 0x77)
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(200)
    k = _randn(g, total, heads, dim) if k is None else k
    v = _randn(g, total, heads, dim) if v is None else v
    api.cache_write(cache, k, v, b.table, b.lens.clamp_min(0), starts)
    return cache, mc.quantised(k, fmt), mc.quantised(v, fmt)


def _expect(b, q, k, v, scale, dtype, there=None):
    want = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    at = key = 0
    for s, (n, length) in enumerate(b.sizes):
        size = max(length, 0)
        want[at:at + n], bound[at:at + n] = attention(
            q[at:at + n], k[key:key + size], v[key:key + size], length - n, scale, dtype,
            None if there is None else there[s])
        at, key = at + n, key + size
    return want, bound


def _inside(got, want, bound, what):
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    off = torch.where(nan, torch.zeros_like(want), (got.double() - want).abs())
    bad = off > torch.where(nan, torch.ones_like(bound), bound)
    assert not bool(bad.any()), \
        f"{what}: {int(bad.sum())} outside, worst {float((off / bound).nan_to_num(0).max()):.3g}"


# (new, length) of the sequences: single tokens; a few each; none and empty ones between; chunks on
# their own and behind a history; rows without keys
BATCHES = {
    "one": [(1, 1)],
    "token": [(1, 77)],
    "tokens": [(1, 1), (1, 32), (1, 33), (1, 127), (1, 128), (1, 129), (1, 700)],
    "drafts": [(4, 100), (3, 3), (0, 50), (2, 257), (0, 0), (1, 600)],
    "chunk": [(70, 70)],
    "chunks": [(64, 64), (200, 513), (1, 300), (0, 9), (33, 1000), (17, 17)],
    "both kinds": [(1, 90), (20, 150), (70, 333), (300, 700), (5, 64), (9, 40)],
    "no keys": [(3, 1), (5, 0), (2, -4), (40, 20)],
}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,group,dim,page",
                         [(1, 1, 64, 16), (2, 4, 64, 1), (8, 4, 128, 32), (1, 7, 128, 64),
                          (2, 3, 256, 16), (3, 16, 64, 256), (1, 33, 128, 8)])
def test_attention(heads, group, dim, page, dtype, fmt):
    for n, (name, sizes) in enumerate(BATCHES.items()):
        _say(f"attention {heads}x{group}x{dim} page {page} {dtype} {fmt} {name}")
        g = _gen(n)
        b = Batch(sizes, page, g, extra_rows=3)
        cache, k, v = _fill(b, heads, dim, fmt, g)
        q = _randn(g, b.rows, heads * group, dim).to(dtype)
        want, bound = _expect(b, q, k, v, dim ** -0.5, dtype)
        out = torch.full_like(q, 7.0)
        o = api.cache_attention(q, cache, *b.where, out=out)
        mine = int(b.starts[-1])
        _inside(o[:mine], want[:mine], bound[:mine], name)
        assert bool((o[mine:] == 7).all()), "rows behind the last sequence were written"
        assert torch.equal(o, api.cache_attention(q, cache, *b.where, out=out.clone()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes", [[(1, 6000)], [(300, 9000)], [(1, 5000)] * 3 + [(40, 4100)],
                                   [(2048, 2048)]])
def test_long(sizes, dtype):
    """Sequences whose keys are cut into runs."""
    _say(f"long {sizes} {dtype}")
    g = _gen(len(sizes))
    b = Batch(sizes, 64, g)
    cache, k, v = _fill(b, 2, 128, "fp8", g)
    q = _randn(g, b.rows, 6, 128).to(dtype)
    want, bound = _expect(b, q, k, v, 128 ** -0.5, dtype)
    _inside(api.cache_attention(q, cache, *b.where), want, bound, "long")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [0.01, 3.0])
def test_scale_and_sharp_weights(scale, dtype):
    g = _gen(1)
    b = Batch([(30, 400), (1, 200)], 32, g)
    cache, k, v = _fill(b, 2, 64, "fp8", g)
    q = _randn(g, b.rows, 4, 64).to(dtype)
    want, bound = _expect(b, q, k, v, scale, dtype)
    _inside(api.cache_attention(q, cache, *b.where, scale=scale), want, bound, f"scale {scale}")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("sizes", [[(1, 200)], [(150, 333), (20, 64)], [(5, 2000), (1, 90)]])
def test_every_key_counts_once(sizes, dim, fmt):
    """Keys of zero make every weight one; value t is one in dim t mod D: an output times the
    number of keys is the number of keys seen of that residue."""
    g = _gen(2)
    b = Batch(sizes, 16, g)
    _, total = b.whole()
    t = torch.cat([torch.arange(length, device="cuda") for _, length in sizes])
    v = torch.zeros(total, 2, dim, device="cuda")
    v[torch.arange(total, device="cuda"), :, t % dim] = 1.0
    cache, _, _ = _fill(b, 2, dim, fmt, g, k=torch.zeros(total, 2, dim, device="cuda"), v=v)
    q = _randn(g, b.rows, 6, dim)
    o = api.cache_attention(q, cache, *b.where)
    at = 0
    for n, length in sizes:
        for i in range(n):
            seen = length - n + i + 1
            want = torch.bincount(torch.arange(seen, device="cuda") % dim, minlength=dim).double()
            got = o[at + i].double() * seen
            assert bool(((got - want).abs() <= 2.0 ** -22 * want).all())
        at += n


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes", [[(6, 90)], [(90, 200)]])
def test_nan_reaches_those_who_see_it(sizes, dtype):
    """Key and value groups that stand for NaN, among them in keys that no query or only later
    ones see."""
    g = _gen(3)
    b = Batch(sizes, 16, g)
    n, length = sizes[0]
    for which in ("k", "v", "both"):
        for t in (0, length - n, length - 1, length - n // 2):
            k, v = _randn(g, length, 2, 64), _randn(g, length, 2, 64)
            if which != "v":
                k[t, 1, 5] = NAN
            if which != "k":
                v[t, 0, 40] = float("inf")
            cache, kq, vq = _fill(b, 2, 64, "fp8", g, k=k, v=v)
            q = _randn(g, b.rows, 4, 64).to(dtype)
            want, bound = _expect(b, q, kq, vq, 0.125, dtype)
            _inside(api.cache_attention(q, cache, *b.where), want, bound, f"{which} at {t}")


@pytest.mark.parametrize("dtype", TYPES)
def test_nan_query_stays_alone(dtype):
    g = _gen(4)
    for sizes in ([(1, 50), (3, 60)], [(100, 150)]):
        b = Batch(sizes, 16, g)
        cache, _, _ = _fill(b, 2, 64, "fp4", g)
        q = _randn(g, b.rows, 4, 64).to(dtype)
        clean = api.cache_attention(q, cache, *b.where)
        q[1, 2, 3] = NAN
        o = api.cache_attention(q, cache, *b.where)
        assert bool(torch.isnan(o[1, 2]).all())
        keep = torch.ones(o.shape[:2], dtype=torch.bool, device="cuda")
        keep[1, 2] = False
        assert torch.equal(o[keep], clean[keep])


@pytest.mark.parametrize("sizes", [[(2, 64)], [(50, 64)]])
def test_pages_that_are_not_there(sizes):
    """Pages of -1 and past the cache: their keys are seen by nobody, and nothing is read there."""
    g = _gen(5)
    b = Batch(sizes, 8, g)
    cache, k, v = _fill(b, 2, 64, "fp8", g)
    b.table[0, 1], b.table[0, 4], b.table[0, 7] = -1, b.pages, 2 ** 31 - 1
    there = torch.ones(64, dtype=torch.bool, device="cuda")
    for p in (1, 4, 7):
        there[8 * p:8 * p + 8] = False
    q = _randn(g, b.rows, 4, 64)
    want, bound = _expect(b, q, k, v, 0.125, torch.float32, [there])
    _inside(api.cache_attention(q, cache, *b.where), want, bound, "missing pages")
    b.table.fill_(-1)
    assert float(api.cache_attention(q, cache, *b.where).abs().max()) == 0
    # lengths past the table's width: keys end with it
    b = Batch(sizes, 8, g)
    cache, k, v = _fill(b, 2, 64, "fp8", g)
    b.table = b.table[:, :5].contiguous()
    there = torch.arange(64, device="cuda") < 40
    want, bound = _expect(b, q, k, v, 0.125, torch.float32, [there])
    _inside(api.cache_attention(q, cache, *b.where), want, bound, "short table")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sizes", [[(1, 37), (3, 130)], [(90, 203), (1, 5)]])
def test_places_that_nobody_wrote(sizes, fmt):
    """NaN codes and scale bytes behind the sequences' ends and in pages of no sequence."""
    g = _gen(9)
    b = Batch(sizes, 16, g)
    starts, total = b.whole()
    k, v = _randn(g, total, 2, 128), _randn(g, total, 2, 128)
    q = _randn(g, b.rows, 8, 128).bfloat16()
    got = []
    for code, scale in ((0, 0), (0xFF, 255), (0x7F, 127)):
        cache = api.Cache.empty(b.pages, 2, 16, 128, fmt)
        for t in (cache.k_codes, cache.v_codes):
            t.fill_(code)
        for t in (cache.k_scale, cache.v_scale):
            t.fill_(scale)
        api.cache_write(cache, k, v, b.table, b.lens, starts)
        got.append(api.cache_attention(q, cache, *b.where))
    assert bool(got[0].isfinite().all())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_strides():
    """Queries, outputs and the table as slices of wider tensors."""
    g = _gen(6)
    b = Batch([(9, 40), (1, 70)], 16, g)
    cache, k, v = _fill(b, 2, 128, "fp8", g)
    wide = torch.full((b.rows, 11, 136), NAN, device="cuda", dtype=torch.bfloat16)
    q = wide[:, 2:10, 3:131]
    q.copy_(_randn(g, *q.shape))
    table = torch.full((2, 20), 10 ** 6, dtype=torch.int32, device="cuda")
    table[:, 4:4 + b.table.shape[1]] = b.table
    out = torch.full_like(wide, 5.0)
    o = api.cache_attention(q, cache, table[:, 4:4 + b.table.shape[1]], b.lens, b.starts,
                            out=out[:, 1:9, 7:135])
    assert torch.equal(o, api.cache_attention(q.contiguous(), cache, *b.where))
    o.fill_(5.0)
    assert bool((out == 5).all())


def test_many_sequences():
    """More sequences than one step of the items' search takes."""
    g = _gen(7)
    for seqs in (65, 200):
        sizes = [(s % 3, 1 + (s * 37) % 150) for s in range(seqs)]
        sizes = [(min(n, length), length) for n, length in sizes]
        sizes[seqs // 2] = (60, 140)
        b = Batch(sizes, 16, g)
        cache, k, v = _fill(b, 1, 64, "fp8", g)
        q = _randn(g, b.rows, 4, 64).half()
        want, bound = _expect(b, q, k, v, 0.125, torch.float16)
        _inside(api.cache_attention(q, cache, *b.where), want, bound, f"{seqs} sequences")


@pytest.mark.parametrize("lone", [True, False])
def test_thousands_of_sequences(lone):
    """Items found in running sums over more sequences than one turn of them takes, long ones cut
    into runs among them; single tokens alone, and with chunks."""
    g = _gen(10)
    sizes = [(1 if s % 5 else 0, 1 + s * 37 % 90) for s in range(1100)]
    sizes[3], sizes[1040] = (1, 9000), (1, 4000)
    if not lone:
        sizes[7], sizes[1030], sizes[1099] = (300, 3000), (150, 2000), (40, 40)
    b = Batch(sizes, 16, g)
    cache, k, v = _fill(b, 2, 64, "fp8", g)
    q = _randn(g, b.rows, 8, 64).bfloat16()
    want, bound = _expect(b, q, k, v, 0.125, torch.bfloat16)
    out = api.cache_attention(q, cache, *b.where)
    _inside(out, want, bound, "1100 sequences")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = api.cache_attention(q, cache, *b.where)
    for _ in range(3):
        o.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, out)


def test_workspaces_streams_and_graphs():
    """Two graphs that share a workspace one after the other, another stream, a workspace larger than
    needed, full of NaN."""
    g = _gen(8)
    ws = api.Workspace(_lib.tcq_cache_attention_workspace_bytes(128, 2, 8, 2, 600) + 4096)
    ws.buf.fill_(255)
    runs = []
    for sizes in ([(1, 3000), (1, 500)], [(500, 2500), (1, 40)]):
        b = Batch(sizes, 32, g)
        cache, _, _ = _fill(b, 2, 128, "fp8", g)
        q = _randn(g, b.rows, 8, 128).bfloat16()
        want = api.cache_attention(q, cache, *b.where)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            o = api.cache_attention(q, cache, *b.where, workspace=ws)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(o, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = api.cache_attention(q, cache, *b.where, workspace=ws)
        runs.append((graph, b, q, cache, o))
    for _ in range(3):
        for graph, b, q, cache, o in runs:
            q.copy_(_randn(g, *q.shape))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, api.cache_attention(q, cache, *b.where))


def test_nothing_to_do():
    g = _gen(9)
    b = Batch([(0, 30), (0, 0)], 16, g)
    cache, _, _ = _fill(b, 2, 64, "fp8", g)
    assert api.cache_attention(torch.zeros(0, 4, 64, device="cuda"), cache,
                               *b.where).shape == (0, 4, 64)
    q = torch.zeros(5, 4, 64, device="cuda")
    out = torch.full_like(q, 3.0)
    assert bool((api.cache_attention(q, cache, *b.where, out=out) == 3).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_layer_decodes(dtype):
    """The operators as a served layer uses them: coded projections of the new tokens' rows, keys
    and values into the cache, attention over it, a microscaled output projection; a prompt in
    one chunk, and one in two chunks with tokens behind it, one by one and drafted."""
    import numpy as np
    import linear_check as lc
    heads, group, dim, N, tokens = 2, 4, 64, 512, 90
    L, kk, V, T = 8, 2, 1, 64
    g, rng = _gen(10), np.random.default_rng(0)
    M = (group + 2) * heads * dim
    bits, s0 = lc.random_streams(rng, M * (N // T), L, kk, V, T)
    bits, s0 = (torch.from_numpy(t.view(np.int32)).cuda() for t in (bits, s0))
    table = _randn(g, 1 << L, V).to(dtype)
    scale = torch.full((M,), N ** -0.5, device="cuda")
    wo = api.mx_pack(_randn(g, N, group * heads * dim) * (group * heads * dim) ** -0.5, "fp4")
    x = _randn(g, tokens, N).to(dtype)

    def step(cache, rows, length):
        n = rows.shape[0]
        qkv = api.decode_linear(bits, s0, table, rows, M, N, L, kk, V, T, row_scale=scale)
        qkv = qkv.view(n, (group + 2) * heads, dim)
        where = (pages, torch.tensor([length], dtype=torch.int32, device="cuda"),
                 torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        q, k, v = qkv.split([group * heads, heads, heads], 1)
        api.cache_write(cache, k, v, *where)
        o = api.cache_attention(q, cache, *where)
        y = api.mx_linear(o.view(n, -1), wo, residual=rows, x_format="fp8")
        return y, o, qkv

    pages = torch.randperm(6, generator=g, device="cuda").int().view(1, 6)
    caches = [api.Cache.empty(6, heads, 16, dim) for _ in range(2)]
    wide = api.mx_unpack(wo, torch.float32).double()

    def check(cache, chunks, what):
        parts, at = [], 0
        for n in chunks:
            at += n
            parts.append(step(cache, x[at - n:at], at))
        y, o, qkv = (torch.cat(p) for p in zip(*parts))
        # (projections of few rows and of many may round differently: each against its own)
        q = qkv[:, :group * heads]
        k, v = (mc.quantised(qkv[:, i:i + heads], "fp8")
                for i in (group * heads, (group + 1) * heads))
        _inside(o, *attention(q, k, v, 0, dim ** -0.5, dtype), f"{what}: attention")
        want, mag = mc.linear(mc.quantised(o.reshape(tokens, -1), "fp8"), wide, None, x)
        _inside(y, want, mc.linear_bound(want, mag, None, x, wide.shape[1], dtype),
                f"{what}: projection")

    check(caches[0], (tokens,), "one chunk")
    check(caches[1], (50, 33, 1, 1, 4, 1), "chunks and tokens")
