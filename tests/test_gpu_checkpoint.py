"""8-bit activation checkpoints (tcq_act_pack, tcq_act_unpack) against their definition in
float64: codes, scale bytes and read-back values must be equal, since both directions are
exact but for the one rounding to an integer that the definition names."""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import _lib, api  # noqa: E402

import linear_check as lc  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]


def _say(msg):
    sys.stdout.write(msg + "\n")
    sys.stdout.flush()


def _values(rng, rows, cols, kind):
    x = rng.standard_normal((rows, cols))
    if kind == "spread":  # groups of very different sizes
        x *= np.exp2(rng.integers(-20, 12, size=(rows, 1)).astype(float))
    elif kind == "ties":  # multiples of half a step around every magnitude
        x = rng.integers(-255, 256, size=(rows, cols)) / 2.0
    elif kind == "zeros":
        x[rng.random((rows, cols)) < 0.9] = 0.0
        x[::2] = 0.0
    return x


def _check(x):
    p = api.act_pack(x)
    back = api.act_unpack(p, x.dtype)
    torch.cuda.synchronize()
    codes, scale = lc.pack(x)
    assert np.array_equal(p.scale.cpu().numpy(), scale)
    assert np.array_equal(p.codes.cpu().numpy(), codes)
    want = torch.from_numpy(lc.unpack(codes, scale)).to(x.dtype).cuda()
    assert torch.equal(torch.nan_to_num(back, nan=77.0), torch.nan_to_num(want, nan=77.0))
    wide = api.act_unpack(p, torch.float32)
    assert torch.equal(torch.nan_to_num(wide.double(), nan=77.0),
                       torch.nan_to_num(torch.from_numpy(lc.unpack(codes, scale)).cuda(),
                                        nan=77.0))
    return p, back


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (2, 32), (3, 33), (5, 64), (7, 100),
                                       (130, 257), (64, 2048), (3, 14336), (1000, 40)])
def test_pack_matches_definition(rows, cols, dtype):
    rng = np.random.default_rng(rows * 7 + cols)
    for kind in ("normal", "spread", "ties", "zeros"):
        _say(f"checkpoint {rows}x{cols} {dtype} {kind}")
        _check(torch.from_numpy(_values(rng, rows, cols, kind)).to(dtype).cuda())


@pytest.mark.parametrize("dtype", TYPES)
def test_error_is_half_a_step(dtype):
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((40, 512))).to(dtype).cuda()
    p, back = _check(x)
    step = torch.ldexp(torch.ones(p.scale.shape, dtype=torch.float64),
                       (p.scale.cpu().int() - 133)).repeat_interleave(32, 1)
    off = (back.double() - x.double()).abs().cpu()
    clamped = p.codes.cpu().int().abs() == 127
    assert bool((off <= torch.where(clamped, step, step / 2)).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_extremes(dtype):
    """The type's largest, smallest normal and smallest subnormal values, zeros of both
    signs; no code's value overflows the type."""
    f = torch.finfo(dtype)
    x = torch.zeros(8, 64, dtype=dtype)
    x[0, 0], x[0, 40] = f.max, -f.max
    x[1, :] = f.max
    x[2, 3], x[2, 4] = f.tiny, f.tiny / 2
    x[3, 0] = f.tiny * f.eps
    x[4, :] = -f.tiny * f.eps
    x[5, :] = -0.0
    x[6, 1], x[6, 2] = 1.0, f.tiny
    _, back = _check(x.cuda())
    assert bool(torch.isfinite(back).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_nonfinite_marks_its_group_alone(dtype):
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((6, 100))).to(dtype)
    x[0, 5], x[1, 40], x[2, 99], x[3, 32] = float("nan"), float("inf"), -float("inf"), \
        float("nan")
    _, back = _check(x.cuda())
    bad = torch.isnan(back).cpu()
    want = torch.zeros(6, 100, dtype=torch.bool)
    want[0, :32], want[1, 32:64], want[2, 96:], want[3, 32:64] = True, True, True, True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_neighbours(dtype):
    """Rows that start anywhere: a column slice of a wider matrix whose other columns are
    NaN; nothing outside rows x cols is written."""
    rng = np.random.default_rng(5)
    for rows, cols, lead, first in [(9, 70, 101, 3), (4, 64, 96, 8), (1, 5, 9, 1)]:
        wide = torch.full((rows, lead), float("nan"), dtype=dtype)
        wide[:, first:first + cols] = torch.from_numpy(rng.standard_normal((rows, cols))).to(dtype)
        x = wide.cuda()[:, first:first + cols]
        p, _ = _check(x)
        # through the C ABI into buffers with guard columns
        ldq, groups = cols + 5, -(-cols // 32)
        codes = torch.full((rows, ldq), 99, dtype=torch.int8, device="cuda")
        scale = torch.full((rows * groups + 8,), 99, dtype=torch.uint8, device="cuda")
        s = torch.cuda.current_stream().cuda_stream
        dt = api._DTYPES[dtype]
        _lib.tcq_act_pack(x.data_ptr(), dt, rows, cols, x.stride(0), codes.data_ptr(), ldq,
                          scale.data_ptr(), s)
        out = torch.full((rows, cols + 3), 5.0, dtype=dtype, device="cuda")
        _lib.tcq_act_unpack(codes.data_ptr(), ldq, scale.data_ptr(), rows, cols, dt,
                            out.data_ptr(), cols + 3, s)
        torch.cuda.synchronize()
        assert torch.equal(codes[:, :cols], p.codes)
        assert bool((codes[:, cols:] == 99).all()) and bool((scale[rows * groups:] == 99).all())
        assert torch.equal(out[:, :cols], api.act_unpack(p, dtype))
        assert bool((out[:, cols:] == 5.0).all())


def test_empty_and_large():
    for shape in [(0, 5), (5, 0), (0, 0)]:
        p = api.act_pack(torch.empty(shape, device="cuda"))
        assert api.act_unpack(p, torch.float32).shape == shape
    # more than 2^31 bytes of values: offsets pass 32 bits
    rows, cols = 70000, 16384
    _say("checkpoint 70000x16384")
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator("cuda").manual_seed(1))
    p = api.act_pack(x)
    back = api.act_unpack(p, x.dtype)
    for r in (0, rows // 2, rows - 1):
        codes, scale = lc.pack(x[r:r + 1])
        assert np.array_equal(p.codes[r:r + 1].cpu().numpy(), codes)
        assert np.array_equal(p.scale[r:r + 1].cpu().numpy(), scale)
        want = torch.from_numpy(lc.unpack(codes, scale)).to(x.dtype)
        assert torch.equal(back[r:r + 1].cpu(), want)
