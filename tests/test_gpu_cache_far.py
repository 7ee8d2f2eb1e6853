"""A cache whose codes and scale bytes lie past 4 GiB: tokens in its last pages are written, read back
and attended to like those of a small cache."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import api  # noqa: E402

from cache_check import Batch  # noqa: E402


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


# codes past 4 GiB, and scale bytes too
@pytest.mark.parametrize("pages,fmt", [(40000, "fp8"), (1100000, "fp4")])
def test_last_pages(pages, fmt):
    sys.stdout.write(f"far cache of {pages} pages {fmt}\n")
    sys.stdout.flush()
    heads, page, dim = 8, 64, 256
    width = dim if fmt == "fp8" else dim // 2
    per = heads * page * width
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 2 * pages * (per + heads * page * dim // 32) + (8 << 30):
        pytest.skip("not enough memory")
    g = torch.Generator(device="cuda").manual_seed(1)
    b = Batch([(1, 300), (70, 200), (3, 64)], page, g)
    starts, total = b.whole()
    k = torch.randn(total, heads, dim, generator=g, device="cuda")
    v = torch.randn(total, heads, dim, generator=g, device="cuda")
    q = torch.randn(b.rows, heads * 4, dim, generator=g, device="cuda").bfloat16()
    near = api.Cache.empty(b.pages, heads, page, dim, fmt)
    api.cache_write(near, k, v, b.table, b.lens, starts)
    want = (*api.cache_read(near, b.table, b.lens, starts, total, torch.float32),
            api.cache_attention(q, near, *b.where))
    far = api.Cache(*(torch.empty((pages, heads, page, w), dtype=torch.uint8, device="cuda")
                      for w in (width, dim // 32, width, dim // 32)), fmt)
    table = torch.where(b.table >= 0, pages - 1 - b.table, b.table)
    api.cache_write(far, k, v, table, b.lens, starts)
    got = (*api.cache_read(far, table, b.lens, starts, total, torch.float32),
           api.cache_attention(q, far, table, b.lens, b.starts))
    for x, y in zip(got, want):
        assert torch.equal(x, y)
