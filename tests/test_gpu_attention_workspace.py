"""One workspace, sized for the largest batch, for every smaller batch of the attention over the
paged cache, and of the microscaled layer's gradients."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import _lib, api  # noqa: E402

from cache_check import Batch  # noqa: E402


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def test_attention_of_smaller_batches():
    g = _gen(1)
    seqs, rows, dim = 80, 96, 128
    n = _lib.tcq_cache_attention_workspace_bytes(dim, 2, 8, seqs, rows)
    guard = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = api.Workspace(n)
    ws.buf = guard[:n]
    # as many rows in one sequence, in some, one to each, with none
    for sizes in ([(96, 2000)], [(90, 300), (1, 5000), (5, 9)], [(1, 30 + s) for s in range(80)],
                  [(1, 70)], [(0, 12), (3, 400)], [(40, 100)] + [(1, 50)] * 50):
        b = Batch(sizes, 16, g)
        cache = api.Cache.empty(b.pages, 2, 16, dim)
        starts, total = b.whole()
        api.cache_write(cache, _randn(g, total, 2, dim), _randn(g, total, 2, dim), b.table, b.lens,
                        starts)
        q = _randn(g, b.rows, 8, dim).bfloat16()
        want = api.cache_attention(q, cache, *b.where)
        assert torch.equal(api.cache_attention(q, cache, *b.where, workspace=ws), want)
        assert bool((guard[n:] == 0xA5).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_gradients_of_smaller_batches(dtype):
    g = _gen(2)
    M, N, most = 200, 520, 900
    w = api.mx_pack(_randn(g, M, N), "fp4")
    n = _lib.tcq_mx_linear_backward_workspace_bytes(api._DTYPES[dtype], most, M, N, True, True,
                                                    True)
    guard = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    ws = api.Workspace(n)
    ws.buf = guard[:n]
    for B in (900, 1, 17, 300, 64):
        x, dy = api.mx_pack(_randn(g, B, N), "fp8"), _randn(g, B, M).to(dtype)
        for xs, dx, db in ((x, True, True), (None, True, False), (x, False, True)):
            for a, e in zip(api.mx_linear_backward(dy, w, xs, dx=dx, dbias=db, workspace=ws),
                            api.mx_linear_backward(dy, w, xs, dx=dx, dbias=db)):
                assert (a is None and e is None) or torch.equal(a, e)
        assert bool((guard[n:] == 0xFF).all())
