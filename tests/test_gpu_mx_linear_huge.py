"""The microscaled linear layer over so many codes that one thread to each 16 bytes of them would
be more threads than a launch may have."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import api  # noqa: E402


def test_codes_past_64_gib():
    B, M, N = 65552, 16, 1 << 21
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 200 << 30:
        pytest.skip("not enough memory")
    # row b's codes all stand for one of 0, 1/2, .., 6 (and so do W's), one group of it for another
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    b = torch.arange(B, device="cuda")
    one, other, at = b % 8, (b // 8) % 8, (b * 7919) % (N // 32)
    codes = torch.empty(B, N // 2, dtype=torch.uint8, device="cuda")
    codes.copy_((one * 17).to(torch.uint8)[:, None].expand(-1, N // 2))
    codes.view(B, N // 32, 16)[b, at] = (other * 17).to(torch.uint8)[:, None]
    x = api.MxPacked(codes, torch.full((B, N // 32), 127, dtype=torch.uint8, device="cuda"), N,
                     "fp4")
    r = torch.arange(M, device="cuda") % 8
    w = api.MxPacked((r * 17).to(torch.uint8)[:, None].expand(-1, N // 2).contiguous(),
                     torch.full((M, N // 32), 125, dtype=torch.uint8, device="cuda"), N, "fp4")
    y = api.mx_linear(x, w, dtype=torch.float32)
    # (32 products to a group, multiples of 1/16: groups' sums are multiples of 2 up to 9 x 2^21 in
    # all, so that every sum is an fp32 number)
    want = (grid[one] * (N - 32) + grid[other] * 32)[:, None] * grid[r][None, :] / 4
    assert torch.equal(y.double(), want)
    del x, codes, y
    torch.cuda.empty_cache()
