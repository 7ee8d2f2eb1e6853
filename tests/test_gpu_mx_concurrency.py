"""Several host threads, each on its own stream, call the microscaled layer, the cache and the
attention over it at the same time: the results are bitwise those of the calls one after another."""
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import api  # noqa: E402

from cache_check import Batch  # noqa: E402

# (rows of x, its format, rows and columns of W; sequences, dim): few and many rows, LDS of several
# sizes
PROBLEMS = [(3, "fp8", 260, 512, [(1, 900), (1, 30)], 64), (120, "fp4", 300, 640, [(70, 300)], 128),
            (600, "fp4", 2000, 700, [(1, 60 + s) for s in range(70)], 128),
            (700, "fp8", 200, 384, [(100, 2000), (2, 50)], 256)]


def _make(i):
    rows, fmt, M, N, sizes, dim = PROBLEMS[i]
    g = torch.Generator(device="cuda").manual_seed(i)
    r = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    b = Batch(sizes, 16, g)
    starts, total = b.whole()
    return (fmt, api.mx_pack(r(M, N), "fp4"), r(rows, N).bfloat16(), b, starts,
            api.Cache.empty(b.pages, 2, 16, dim), r(total, 2, dim), r(total, 2, dim),
            r(b.rows, 8, dim).bfloat16())


def _run(fmt, w, x, b, starts, cache, k, v, q):
    y, kept = api.mx_linear(x, w, x_format=fmt, keep=True)
    api.cache_write(cache, k, v, b.table, b.lens, starts)
    o = api.cache_attention(q, cache, *b.where)
    return [y, *api.mx_linear_backward(y, w, kept), o,
            *api.cache_read(cache, b.table, b.lens, starts, k.shape[0], torch.float32)]


def test_threads_on_own_streams():
    problems = [_make(i) for i in range(len(PROBLEMS))]
    want = [[t.clone() for t in _run(*p)] for p in problems]
    torch.cuda.synchronize()
    got, errors = [None] * len(problems), []
    start = threading.Barrier(len(problems))

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                start.wait(timeout=60)
                for _ in range(5):
                    got[i] = _run(*problems[i])
                s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(problems))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=100)
    assert not errors, errors
    for a, b in zip(got, want):
        assert a is not None
        for x, y in zip(a, b):
            assert torch.equal(x, y)
