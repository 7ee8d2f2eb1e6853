"""The microscaled linear layer over codes whose rows lie so far apart that a tile of them spans
more than 4 GiB, or nearly: the same as over rows without gaps."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import api  # noqa: E402


def _grid(g, rows, cols):
    """Values on a grid on which every partial sum is an fp32 number."""
    v = torch.randint(-3, 4, (rows, cols), generator=g, device="cuda").float()
    v[:, ::32] = 4.0
    e = torch.randint(-1, 2, (rows, -(-cols // 32)), generator=g, device="cuda").float()
    return v * torch.exp2(e).repeat_interleave(32, 1)[:, :cols]


def _far(p, pitch):
    """p with rows of codes `pitch` bytes apart, the bytes between them codes of 6."""
    rows, width = p.codes.shape
    flat = torch.empty(rows * pitch, dtype=torch.uint8, device="cuda")
    wide = flat.view(rows, pitch)
    near = min(4096, pitch)
    wide[:, :near] = 0x77
    codes = wide[:, 64:64 + width]
    codes.copy_(p.codes)
    assert codes.stride(0) == pitch
    return api.MxPacked(codes, p.scale, p.cols, p.format)


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


# tiles of 256 and of 128 rows; the last pitch that a tile's 32-bit offsets hold and those past it
@pytest.mark.parametrize("pitch", [1 << 24, (1 << 24) + 16, 16843024, 1 << 25, (1 << 25) + (1 << 19)])
@pytest.mark.parametrize("B,M", [(16384, 272), (6800, 272)])
def test_matrix(B, M, pitch):
    sys.stdout.write(f"far matrix {B}x{M} pitch {pitch}\n")
    sys.stdout.flush()
    g = torch.Generator(device="cuda").manual_seed(pitch % 1000)
    N = 200
    x, w = _grid(g, B, N), api.mx_pack(_grid(g, M, N), "fp4")
    bias = torch.randint(-9, 9, (M,), generator=g, device="cuda").float()
    want = api.mx_linear(x, w, bias=bias, x_format="fp4")
    exact = api.mx_unpack(api.mx_pack(x, "fp4"), torch.float32).double() @ \
        api.mx_unpack(w, torch.float32).double().t().contiguous() + bias
    assert torch.equal(want.double(), exact)
    far = _far(w, pitch)
    assert torch.equal(api.mx_linear(x, far, bias=bias, x_format="fp4"), want)
    y, kept = api.mx_linear(x, far, bias=bias, residual=want, x_format="fp4", keep=True)
    p = api.mx_pack(x, "fp4")
    assert torch.equal(kept.codes, p.codes) and torch.equal(kept.scale, p.scale)
    assert torch.equal(y.double(), 2 * exact)


@pytest.mark.parametrize("pitch", [1 << 24, 16843024, (1 << 25) + (1 << 19)])
@pytest.mark.parametrize("B,M", [(300, 16400), (290, 4900)])
def test_packed_rows(B, M, pitch):
    sys.stdout.write(f"far rows {B}x{M} pitch {pitch}\n")
    sys.stdout.flush()
    g = torch.Generator(device="cuda").manual_seed(pitch % 1000 + 1)
    N = 321
    x, w = api.mx_pack(_grid(g, B, N), "fp4"), api.mx_pack(_grid(g, M, N), "fp4")
    want = api.mx_linear(x, w, dtype=torch.float32)
    assert torch.equal(api.mx_linear(_far(x, pitch), w, dtype=torch.float32), want)


def test_other_formats_and_calls():
    """8-bit rows, few rows, gradients and unpacking hold such offsets in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(3)
    N, M, pitch = 100, 280, (1 << 24) + 4096
    w = api.mx_pack(_grid(g, M, N), "fp4")
    far = _far(w, pitch)
    assert torch.equal(api.mx_unpack(far, torch.float32), api.mx_unpack(w, torch.float32))
    for B, fmt in ((3, "fp4"), (60, "fp4"), (60, "fp8"), (700, "fp8")):
        x = _grid(g, B, N)
        assert torch.equal(api.mx_linear(x, far, x_format=fmt), api.mx_linear(x, w, x_format=fmt))
    dy = torch.randint(-3, 4, (50, M), generator=g, device="cuda").bfloat16()
    assert torch.equal(api.mx_linear_backward(dy, far)[0], api.mx_linear_backward(dy, w)[0])


def test_pieces_of_a_large_batch():
    """More rows than one launch of the product for far rows takes."""
    g = torch.Generator(device="cuda").manual_seed(4)
    B, M, N = (1 << 19) + 37, 40, 64
    x = api.mx_pack(_grid(g, B, N), "fp4")
    w = api.mx_pack(_grid(g, M, N), "fp4")
    want = api.mx_linear(x, w, dtype=torch.float32)
    res = torch.randint(-9, 9, (B, M), generator=g, device="cuda").float()
    far = _far(w, (1 << 24) + 16)
    assert torch.equal(api.mx_linear(x, far, residual=res, dtype=torch.float32), want + res)
    v = api.mx_unpack(x, torch.float32)
    y, kept = api.mx_linear(v, far, x_format="fp4", keep=True)
    assert torch.equal(y, want) and torch.equal(kept.codes, x.codes) and \
        torch.equal(kept.scale, x.scale)
