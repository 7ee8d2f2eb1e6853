"""The float64 reference of the microscaled formats against hand-computed codes and values."""
import math

import pytest

torch = pytest.importorskip("torch")

import mx_check as mc


def test_tables():
    assert mc.table("fp4").tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    t = mc.table("fp8")
    assert t.numel() == 127 and t[126] == 448 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6
    assert bool((t[1:] > t[:-1]).all())


@pytest.mark.parametrize("value,code", [(0.0, 0), (-0.0, 8), (0.25, 0), (0.26, 1), (0.75, 2),
                                        (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6),
                                        (5.01, 7), (-5.0, 14), (7.9, 7)])
def test_fp4_codes(value, code):
    # 4 fixes the scale at one (exponent field 129, less 2)
    x = torch.full((1, 32), 4.0)
    x[0, 3] = value
    c, e = mc.codes_of(x, "fp4")
    assert e.tolist() == [[127]] and c[0, 3] == code and c[0, 0] == 6


def test_fp8_codes_match_torch():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(64, 256, generator=g) * torch.exp(3 * torch.randn(64, 1, generator=g))
    c, e = mc.codes_of(x, "fp8")
    v = (x.double() * torch.exp2(127.0 - e.double()).repeat_interleave(32, 1)).clamp(-448, 448)
    want = v.float().to(torch.float8_e4m3fn)
    assert torch.equal(mc.table("fp8")[(c & 127).long()] * torch.where(c > 127, -1.0, 1.0),
                       want.double())


def test_special_groups():
    x = torch.zeros(1, 128)
    x[0, 1], x[0, 40], x[0, 70] = math.inf, math.nan, 2.0 ** -140
    for fmt in ("fp4", "fp8"):
        c, e = mc.codes_of(x, fmt)
        assert e.tolist() == [[255, 255, 0, 0]] and c[0, :64].max() == 0
        v = mc.values_of(c, e, fmt)
        assert bool(torch.isnan(v[0, :64]).all()) and not bool(torch.isnan(v[0, 64:]).any())


def test_stored_bytes():
    c = torch.arange(16, dtype=torch.uint8).repeat(2).view(1, 32)
    s = mc.store(c, "fp4")
    assert s[0, 0] == 0x10 and s[0, 7] == 0xFE
    assert torch.equal(mc.load(s, "fp4"), c)
