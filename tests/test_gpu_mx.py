"""Microscaled quantisation (tcq_mx_pack, tcq_mx_unpack) against its definition in float64: codes,
scale bytes and read-back values are equal, since each code has one rounding, which the
definition names, and reading back is exact."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import _lib, api  # noqa: E402

import mx_check as mc  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]
FORMATS = ["fp4", "fp8"]


def _say(msg):
    sys.stdout.write(msg + "\n")
    sys.stdout.flush()


def _same(a, b):
    return torch.equal(torch.nan_to_num(a.double(), nan=77.0, posinf=78.0, neginf=79.0),
                       torch.nan_to_num(b.double(), nan=77.0, posinf=78.0, neginf=79.0))


def _check(x, fmt):
    p = api.mx_pack(x, fmt)
    codes, scale = mc.codes_of(x, fmt)
    assert torch.equal(p.scale, scale)
    assert torch.equal(p.codes, mc.store(codes, fmt))
    v = mc.values_of(codes, scale, fmt)[:, :x.shape[1]]
    for t in TYPES:
        assert _same(api.mx_unpack(p, t), v.to(t)), t
    return p


def _values(g, rows, cols, kind):
    x = torch.randn(rows, cols, generator=g, device="cuda")
    if kind == "spread":  # groups of very different sizes
        x *= torch.exp2(torch.randint(-20, 12, (rows, 1), generator=g, device="cuda").float())
    elif kind == "ties":  # halfway between codes, and on them
        x = torch.randint(-64, 65, (rows, cols), generator=g, device="cuda") / 8.0
    elif kind == "zeros":
        x[torch.rand(rows, cols, generator=g, device="cuda") < 0.9] = 0.0
        x[::2] = 0.0
    return x


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (2, 32), (3, 33), (5, 64), (7, 100),
                                       (130, 257), (64, 2048), (3, 14336), (1000, 40)])
def test_pack_matches_definition(rows, cols, dtype, fmt):
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + cols)
    for kind in ("normal", "spread", "ties", "zeros"):
        _say(f"microscaled {rows}x{cols} {dtype} {fmt} {kind}")
        _check(_values(g, rows, cols, kind).to(dtype), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_code_and_scale(fmt):
    """Every code under every scale byte, against the table."""
    n = 16 if fmt == "fp4" else 256
    one = torch.arange(n, dtype=torch.uint8, device="cuda")
    if fmt == "fp8":
        one[127], one[255] = 0, 0  # NaN codes are never written
    codes = one.repeat(256, 2 if fmt == "fp4" else 1)
    groups = codes.shape[1] // 32
    scale = torch.arange(256, dtype=torch.uint8, device="cuda").view(-1, 1).repeat(1, groups)
    p = api.MxPacked(mc.store(codes, fmt).contiguous(), scale.contiguous(), codes.shape[1], fmt)
    v = mc.values_of(codes, scale, fmt)
    for t in TYPES:
        assert _same(api.mx_unpack(p, t), v.float().to(t)), t


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
def test_extremes(dtype, fmt):
    """The type's largest, smallest normal and smallest subnormal values, zeros of both signs."""
    f = torch.finfo(dtype)
    x = torch.zeros(8, 64, dtype=dtype)
    x[0, 0], x[0, 40] = f.max, -f.max
    x[1, :] = f.max
    x[2, 3], x[2, 4] = f.tiny, f.tiny / 2
    x[3, 0] = f.tiny * f.eps
    x[4, :] = -f.tiny * f.eps
    x[5, :] = -0.0
    x[6, 1], x[6, 2] = 1.0, f.tiny
    p = _check(x.cuda(), fmt)
    assert bool(torch.isfinite(api.mx_unpack(p, dtype)).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
def test_nonfinite_marks_its_group_alone(dtype, fmt):
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(6, 100, generator=g, device="cuda").to(dtype)
    x[0, 5], x[1, 40], x[2, 99], x[3, 32] = float("nan"), float("inf"), -float("inf"), \
        float("nan")
    p = _check(x, fmt)
    want = torch.zeros(6, 100, dtype=torch.bool, device="cuda")
    want[0, :32], want[1, 32:64], want[2, 96:], want[3, 32:64] = True, True, True, True
    assert torch.equal(torch.isnan(api.mx_unpack(p, dtype)), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_neighbours(dtype, fmt):
    """Rows that start anywhere in a wider matrix of NaN, into buffers with guard bytes: nothing
    outside whole groups is written, and codes behind the last column are zeros."""
    g = torch.Generator(device="cuda").manual_seed(5)
    code, size = _lib.TCQ_FP4 if fmt == "fp4" else _lib.TCQ_FP8, 16 if fmt == "fp4" else 32
    for rows, cols, lead, first in [(9, 70, 101, 3), (4, 64, 96, 8), (1, 5, 9, 1)]:
        wide = torch.full((rows, lead), float("nan"), dtype=dtype, device="cuda")
        wide[:, first:first + cols] = torch.randn(rows, cols, generator=g, device="cuda").to(dtype)
        x = wide[:, first:first + cols]
        p = _check(x, fmt)
        groups = -(-cols // 32)
        ldq = groups * size + 16
        codes = torch.full((rows + 1, ldq), 99, dtype=torch.uint8, device="cuda")
        scale = torch.full((rows * groups + 8,), 99, dtype=torch.uint8, device="cuda")
        _lib.tcq_mx_pack(x.data_ptr(), api._DTYPES[dtype], rows, cols, lead, code,
                         codes.data_ptr(), ldq, scale.data_ptr(), None)
        torch.cuda.synchronize()
        assert torch.equal(codes[:rows, :groups * size], p.codes)
        assert bool((codes[:, groups * size:] == 99).all()) and bool((codes[rows] == 99).all())
        assert bool((scale[rows * groups:] == 99).all())
        if cols % 32:
            last = mc.load(p.codes[:, (groups - 1) * size:], fmt)
            assert bool((last[:, cols % 32:] == 0).all())
        out = torch.full((rows + 1, lead), 7.0, dtype=dtype, device="cuda")
        _lib.tcq_mx_unpack(codes.data_ptr(), ldq, scale.data_ptr(), rows, cols, code,
                           api._DTYPES[dtype], out[:, first:].data_ptr(), lead, None)
        torch.cuda.synchronize()
        assert torch.equal(out[:rows, first:first + cols], api.mx_unpack(p, dtype))
        assert bool((out[:, :first] == 7).all()) and bool((out[rows] == 7).all())
        assert bool((out[:, first + cols:] == 7).all())


def test_offsets_past_32_bits():
    """A matrix of more than 2^32 bytes and 2^31 values: its last rows are right."""
    rows, cols = 70000, 32768 + 32
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(6)
    tail = torch.randn(3, cols, generator=g, device="cuda").bfloat16()
    x[-3:] = tail
    p = api.mx_pack(x, "fp8")
    codes, scale = mc.codes_of(tail, "fp8")
    assert torch.equal(p.codes[-3:], codes) and torch.equal(p.scale[-3:], scale)
    assert int(p.codes[:-3].max()) == 0
    back = api.mx_unpack(p, torch.bfloat16)
    assert torch.equal(back[-3:].double(), mc.values_of(codes, scale, "fp8"))
    assert float(back[:-3].abs().max()) == 0.0


def test_empty():
    for shape in [(0, 64), (5, 0), (0, 0)]:
        p = api.mx_pack(torch.zeros(shape, device="cuda"), "fp4")
        assert api.mx_unpack(p, torch.float16).shape == shape


def test_another_stream_and_graph():
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(64, 300, generator=g, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p = api.mx_pack(x, "fp4")
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(p.codes, mc.store(mc.codes_of(x, "fp4")[0], "fp4"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = api.mx_pack(x, "fp8")
        back = api.mx_unpack(q, torch.float32)
    for i in range(3):
        x.copy_(torch.randn(64, 300, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(back.double(), mc.quantised(x, "fp8"))
