"""An infinity in a query: every score of its row is one, or NaN, and softmax of either is NaN,
also where all of them are -inf; rows without keys stay zeros."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import api  # noqa: E402

from cache_check import Batch  # noqa: E402

INF = float("inf")


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("sizes", [[(1, 1)], [(1, 700), (3, 40)], [(1, 6000)], [(70, 70)],
                                   [(100, 2000), (1, 9)]])
def test_infinite_query(sizes, dim, dtype):
    g = torch.Generator(device="cuda").manual_seed(dim)
    b = Batch(sizes, 16, g)
    starts, total = b.whole()
    k = torch.randn(total, 2, dim, generator=g, device="cuda")
    v = torch.randn(total, 2, dim, generator=g, device="cuda")
    k[:, :, 5] = -k[:, :, 5].abs() - 1.0   # scores of -inf for q[5] = inf
    cache = api.Cache.empty(b.pages, 2, 16, dim)
    api.cache_write(cache, k, v, b.table, b.lens, starts)
    q = torch.randn(b.rows, 8, dim, generator=g, device="cuda").to(dtype)
    clean = api.cache_attention(q, cache, *b.where)
    assert bool(clean.isfinite().all())
    for row, head, value in ((0, 1, INF), (b.rows - 1, 6, -INF), (b.rows // 2, 3, INF)):
        x = q.clone()
        x[row, head, 5] = value
        o = api.cache_attention(x, cache, *b.where)
        assert bool(o[row, head].isnan().all()), (row, head, value)
        o[row, head] = clean[row, head]
        assert torch.equal(o, clean)
    # a row that sees no key
    x = q.clone()
    x[0, 0, 5] = INF
    b.table.fill_(-1)
    assert float(api.cache_attention(x, cache, *b.where).abs().max()) == 0
