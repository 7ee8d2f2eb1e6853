"""Argument checks of the paged cache and the attention over it: bad calls are rejected before
anything reaches a GPU (no device work is issued by these tests)."""
import ctypes

import pytest

import trellis_coded_bit_amd as tcq
from trellis_coded_bit_amd import _lib

E = _lib
FAKE = 0x7F0000001000  # never dereferenced: every call below fails validation or has no work
FAR = 1 << 36          # apart from one another
BIG = 1 << 45


def _cache(**kw):
    a = dict(k_codes=FAKE, k_scale=FAKE + FAR, v_codes=FAKE + 2 * FAR, v_scale=FAKE + 3 * FAR,
             pages=10, heads=2, page=16, dim=64, format=E.TCQ_FP8)
    a.update({n: v for n, v in kw.items() if n in a})
    return _lib.TcqCache(*a.values())


def _batch(**kw):
    a = dict(table=FAKE + 4 * FAR, ldt=5, width=5, lens=FAKE + 5 * FAR, starts=FAKE + 6 * FAR,
             seqs=3)
    a.update({n: v for n, v in kw.items() if n in a})
    return _lib.TcqCacheBatch(*a.values())


def _move(fn, **kw):
    a = dict(dtype=E.TCQ_BF16, k=FAKE + 7 * FAR, k_row=128, k_head=64, v=FAKE + 8 * FAR, v_row=128,
             v_head=64, rows=0)
    a.update({n: v for n, v in kw.items() if n in a})
    return fn(_cache(**kw), _batch(**kw), *a.values(), None)


def _attend(**kw):
    a = dict(dtype=E.TCQ_BF16, q=FAKE + 7 * FAR, q_row=512, q_head=64, q_heads=8, rows=4,
             scale=0.125, o=FAKE + 8 * FAR, o_row=512, o_head=64, ws=None, wsb=BIG)
    a.update({n: v for n, v in kw.items() if n in a})
    return _lib.load().tcq_cache_attention(_cache(**kw), _batch(**kw), *a.values(), None)


BAD = [dict(format=2), dict(format=-1), dict(dtype=3), dict(pages=-1), dict(heads=0),
       dict(page=0), dict(page=24), dict(k_codes=None), dict(v_scale=None),
       dict(v_codes=FAKE + 2 * FAR + 8), dict(seqs=-1), dict(width=-1), dict(rows=-1),
       dict(ldt=4), dict(lens=None), dict(starts=None), dict(table=None),
       dict(starts=FAKE + 6 * FAR + 2)]
UNSUPPORTED = [dict(dim=32), dict(dim=96), dict(dim=512), dict(heads=1025, k_row=1 << 20),
               dict(page=8192), dict(pages=1 << 31), dict(seqs=(1 << 20) + 1),
               dict(rows=(1 << 23) + 1), dict(width=1 << 31, ldt=1 << 32)]


@pytest.mark.parametrize("name", ["tcq_cache_write", "tcq_cache_read"])
def test_move_argument_checks(name):
    fn = getattr(_lib.load(), name)
    assert _move(fn) == E.TCQ_OK
    for kw in BAD:
        assert _move(fn, **kw) == E.TCQ_EINVAL, kw
        assert name in tcq.tcq_last_error()
    for kw in UNSUPPORTED:
        assert _move(fn, **kw) == E.TCQ_EUNSUPPORTED, kw
    for kw in (dict(k=None), dict(v=None), dict(k=FAKE + 1), dict(k_row=127), dict(k_head=63),
               dict(v_row=100), dict(k=FAKE), dict(v=FAKE + FAR),
               dict(v=FAKE + 3 * FAR + 10 * 2 * 16 * 2 - 2)):
        assert _move(fn, rows=4, **kw) == E.TCQ_EINVAL, kw
    assert _move(fn, rows=4, seqs=0, k=None) == E.TCQ_OK
    assert fn(None, _batch(), 0, FAKE, 128, 64, FAKE, 128, 64, 1, None) == E.TCQ_EINVAL
    assert fn(_cache(), None, 0, FAKE, 128, 64, FAKE, 128, 64, 1, None) == E.TCQ_EINVAL


def test_read_keeps_outputs_apart():
    fn = _lib.load().tcq_cache_read
    for kw in (dict(k=FAKE + 8 * FAR), dict(k=FAKE + 4 * FAR), dict(v=FAKE + 5 * FAR),
               dict(v=FAKE + 6 * FAR)):
        assert _move(fn, rows=4, **kw) == E.TCQ_EINVAL, kw
        assert "overlap" in tcq.tcq_last_error()


def test_attention_argument_checks():
    assert _attend() == E.TCQ_EWORKSPACE
    assert _attend(ws=FAKE, wsb=256) == E.TCQ_EWORKSPACE
    assert _attend(ws=FAKE + 8) == E.TCQ_EINVAL
    for kw in BAD:
        assert _attend(**kw) == E.TCQ_EINVAL, kw
    for kw in UNSUPPORTED:
        assert _attend(**kw) == E.TCQ_EUNSUPPORTED, kw
    for kw in (dict(q=None), dict(o=None), dict(q=FAKE + 1), dict(q_row=511), dict(q_head=63),
               dict(o_row=511), dict(o_head=0), dict(q_heads=7), dict(q_heads=0),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(scale=1e-30)):
        assert _attend(**kw) == E.TCQ_EINVAL, kw
    assert _attend(q_heads=1026, q_row=1 << 20, o_row=1 << 20) == E.TCQ_EUNSUPPORTED
    assert _attend(rows=1 << 22, q_heads=128, q_row=1 << 20, o_row=1 << 20) == E.TCQ_EUNSUPPORTED
    for at in (0, 1, 2, 3, 4, 5, 6, 7):
        assert _attend(o=FAKE + at * FAR, ws=FAKE + 20 * FAR) == E.TCQ_EINVAL
        assert "overlap" in tcq.tcq_last_error()
    assert _attend(rows=0) == E.TCQ_OK and _attend(seqs=0) == E.TCQ_OK


def test_workspace_query():
    lib = _lib.load()
    b = ctypes.c_size_t(1)
    ref = ctypes.byref(b)
    fn = lib.tcq_cache_attention_workspace_bytes
    assert fn(64, 2, 8, 3, 0, ref) == E.TCQ_OK and b.value == 0
    assert fn(64, 2, 8, 3, 5, None) == E.TCQ_EINVAL
    assert fn(64, 2, 7, 3, 5, ref) == E.TCQ_EINVAL
    assert fn(96, 2, 8, 3, 5, ref) == E.TCQ_EUNSUPPORTED
    assert fn(64, 2, 8, -1, 5, ref) == E.TCQ_EUNSUPPORTED
    assert fn(64, 2, 8, 3, 5, ref) == E.TCQ_OK and 0 < b.value < 1 << 30


def test_python_calls_check_their_tensors():
    torch = pytest.importorskip("torch")
    from trellis_coded_bit_amd import api
    cache = api.Cache.empty(4, 2, 16, 64, "fp4", device="cpu")
    assert cache.dim == 64 and cache.k_codes.shape == (4, 2, 16, 32)
    c = cache.c(torch.device("cpu"))
    assert (c.pages, c.heads, c.page, c.dim, c.format) == (4, 2, 16, 64, E.TCQ_FP4)
    k = torch.zeros(3, 2, 64)
    table = torch.zeros(1, 4, dtype=torch.int32)
    lens, starts = torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(AssertionError):
        api.cache_write(cache, k, k, table, lens, starts)  # not on a GPU
    with pytest.raises(AssertionError):
        api._batch(table.long(), lens, starts, torch.device("cpu"))
    with pytest.raises(AssertionError):
        api._batch(table, lens, starts[:1], torch.device("cpu"))
    with pytest.raises(AssertionError):
        api._vectors(k.transpose(1, 2), "k", 3, 64, 2, torch.float32, torch.device("cpu"))
    with pytest.raises(AssertionError):
        api.Cache(cache.k_codes, cache.k_scale, cache.v_codes, cache.v_scale, "fp8").c(
            torch.device("cpu"))
