"""How precisely the coded linear layer's sums are held, against float64: each output within
a bound that counts the roundings which the header's contract names, no others."""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import api  # noqa: E402

import linear_check as lc  # noqa: E402
from test_gpu_linear import Coded, _grad_reference  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _say(msg):
    sys.stdout.write(msg + "\n")
    sys.stdout.flush()


def _scaled(w, factor):
    """The matrix with every table value times a power of two (exact in range)."""
    w.table = (w.table.double() * factor).to(w.table.dtype)
    w.W = w.W * factor
    return w


def _gradients(w, dy, a, act, z, x, dtype):
    """Worst error / bound of dx and dw.  s = dy act'(z) a comes from fp32 steps and is held
    in two terms of the type: half(t)^2 of its value, in fp16 not below 2^-34 of the largest
    row scale (1/2 for none).  Each sum then has two products per term."""
    M, B = w.shape[0], dy.shape[0]
    zp, xp = api.act_pack(z), api.act_pack(x)
    z, x = api.act_unpack(zp, F32).double(), api.act_unpack(xp, F32).double()
    g, s, gx, gw = _grad_reference(w, dy, a, act, z, x, dtype, False)
    dx, dw, db = w.backward(dy, row_scale=a, act=act, z=zp, x=xp)
    torch.cuda.synchronize()
    ra = torch.ones(M, device="cuda", dtype=torch.float64) if a is None else a.double().abs()
    es = dy.double().abs() * lc.slope_error(z, act) * ra + 4 * lc.U * s.abs()
    es = es + lc.half(dtype) ** 2 * (s.abs() + es)
    es = es + (2.0 ** -34 * float(ra.max()) if dtype == F16 else lc.tiny(dtype))
    out = []
    for got, want, left, right, K in ((dx, gx, (s, es), w.W.abs(), M),
                                      (dw, gw, (s.t(), es.t()), x.abs(), B)):
        mag, err = left[0].abs() @ right, left[1] @ right
        lim = err + lc.gamma(2 * K + 2) * (mag + err)
        lim = lim + lc.half(dtype) * (want.abs() + lim) + lc.tiny(dtype)
        out.append(float(((got.double() - want).abs() / lim).nan_to_num(nan=9e9).max()))
    return out


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("L,k,V,T,M,N,B", [
    (16, 2, 1, 256, 130, 512, 37), (8, 2, 1, 64, 21, 64, 3), (16, 2, 1, 256, 1024, 1024, 509),
    (16, 2, 2, 256, 1031, 1024, 1025), (16, 1, 1, 17, 70, 17 * 9, 200)])
def test_gradients_are_rounded_at_the_end(L, k, V, T, M, N, B, act, dtype):
    """16-bit gradients are off by their own rounding alone: what the products read holds
    dy act'(z) row_scale in more bits than the type has."""
    rng = np.random.default_rng(M + B)
    w = Coded(N + B, M, N, L, k, V, T, dtype, False)

    def normal(*size):
        return torch.from_numpy(rng.standard_normal(size)).to(dtype).cuda()
    a = torch.from_numpy(rng.standard_normal(M) / np.sqrt(N)).float().cuda()
    for scale in (a, None):
        r = _gradients(w, normal(B, M), scale, act, normal(B, M), normal(B, N), dtype)
        _say(f"gradients M={M} N={N} B={B} {act} {dtype} row_scale={scale is not None}: "
             f"worst error / bound dx {r[0]:.3g}, dw {r[1]:.3g}")
        assert max(r) <= 1


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rms", [1e-3, 1e-4, 1e-5, 1e-6])
def test_gradients_of_small_dy(rms, dtype):
    """dy far below 1 with a row scale of 1/64: dy is a number of the type, and its product
    with the row scale must not lose what dy has."""
    M, N, B = 512, 512, 300
    rng = np.random.default_rng(5)
    w = Coded(3, M, N, 16, 2, 1, 256, dtype, False)

    def normal(*size):
        return torch.from_numpy(rng.standard_normal(size)).cuda()
    a = torch.from_numpy((1 + rng.random(M)) / 64).float().cuda()
    dy = (normal(B, M) * rms).to(dtype)
    r = _gradients(w, dy, a, "silu", normal(B, M).to(dtype), normal(B, N).to(dtype), dtype)
    _say(f"small dy {rms} {dtype}: worst error / bound dx {r[0]:.3g}, dw {r[1]:.3g}")
    assert max(r) <= 1


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("case", ["row scale", "slope", "both", "tiny row scale"])
def test_gradients_of_large_products(case, dtype):
    """dy act'(z) row_scale past fp16's largest number, with outputs inside its range."""
    M, N, B = 96, 256, 140
    rng = np.random.default_rng(7)
    w = _scaled(Coded(4, M, N, 16, 2, 1, 256, dtype, False), 2.0 ** -9)

    def normal(*size):
        return torch.from_numpy(rng.standard_normal(size)).cuda()
    a, act = None, "gelu"
    dy, z = normal(B, M) * 8, normal(B, M)
    if case in ("row scale", "both"):
        a = torch.from_numpy(rng.standard_normal(M) * 3000).float().cuda()
        dy = dy * 4
    if case == "slope":
        dy, z = 65504 * torch.sign(dy), z * 0 + 1.5     # slope 1.13
    if case == "both":
        dy[3, 4], z[3, 4] = 65504, 1.5
        a[4] = 2.0
    if case == "tiny row scale":
        w = _scaled(w, 2.0 ** 18)
        a = torch.from_numpy(rng.standard_normal(M) * 2.0 ** -20).float().cuda()
    x = (normal(B, N) * 2.0 ** -9).to(dtype)
    r = _gradients(w, dy.to(dtype), a, act, z.to(dtype), x, dtype)
    _say(f"large {case} {dtype}: worst error / bound dx {r[0]:.3g}, dw {r[1]:.3g}")
    assert max(r) <= 1


def test_gradients_of_odd_row_scales():
    """A row scale of zeros, one with an infinity or a NaN in one row, one of subnormals:
    the other rows' gradients are those of the formula."""
    M, N, B = 70, 256, 20
    rng = np.random.default_rng(11)
    for dtype in (F16, BF16):
        w = Coded(6, M, N, 16, 2, 1, 256, dtype, False)
        dy = torch.from_numpy(rng.standard_normal((B, M))).to(dtype).cuda()
        x = torch.from_numpy(rng.standard_normal((B, N))).to(dtype).cuda()
        xp = api.act_pack(x)
        dx, dw, _ = w.backward(dy, row_scale=torch.zeros(M, device="cuda"), x=xp)
        assert bool((dx == 0).all()) and bool((dw == 0).all())
        a = torch.from_numpy(rng.standard_normal(M)).float().cuda()
        a[9] = 0.25  # not the largest
        want = w.backward(dy, row_scale=a, x=xp)[1]
        for bad in (float("inf"), float("-inf"), float("nan")):
            b = a.clone()
            b[9] = bad
            dw = w.backward(dy, row_scale=b, x=xp)[1]
            assert not bool(torch.isfinite(dw[9]).any())
            rows = torch.arange(M, device="cuda") != 9
            assert torch.equal(dw[rows], want[rows])
        small = torch.full((M,), 2.0 ** -140, device="cuda")
        dx, dw, _ = w.backward(dy, row_scale=small, x=xp)
        assert bool((dx.double().abs() <= 2.0 ** -120).all())
        assert bool((dw.double().abs() <= 2.0 ** -120).all())
