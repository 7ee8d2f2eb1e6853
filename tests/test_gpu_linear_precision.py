"""How precisely the coded linear layer's sums are held, against float64: each output within
a bound that counts the roundings which the header's contract names, no others."""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import _lib, api  # noqa: E402

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


# M, N, B whose fp32 products take 64 x 128 tiles, 128 x 128 ones, and both with k split; a
# generic decode before them
F32_SIZES = [(16, 2, 1, 256, 130, 512, 300), (16, 2, 1, 256, 2047, 2048, 1001),
             (16, 2, 1, 256, 4096, 1024, 1100), (8, 1, 1, 20, 300, 500, 140)]


def _f32_table(w, values):
    """The layer with a table of its own and its float64 matrix."""
    w.table = values.to(F32).contiguous()
    M, N, L, k, V, T = w.shape
    w.W = api.decode(w.bits, w.s0, w.table, M, N, L, k, V, T).double()
    return w


@pytest.mark.parametrize("L,k,V,T,M,N,B", F32_SIZES)
def test_f32_single_products(L, k, V, T, M, N, B):
    """One product per output, of numbers whose significands are full of ones or random: left
    out is less than (1 + 2^-9) 2^-23 of it, and of its three orders of partial sums (2^-13,
    2^-6 and 1 of it) each may lose a whole unit of 2^-23."""
    lim = 2.0 ** -23 * (2 + 2.0 ** -9 + 2.0 ** -6 + 2.0 ** -13)
    rng = np.random.default_rng(M)
    w = Coded(M + B, M, N, L, k, V, T, F32, False)

    def ones(*size):
        # 1.0000000 1111111 11111111 in binary and neighbours, random ones among them
        u = np.where(rng.random(size) < 0.5, 0x3F80FFFF - rng.integers(0, 3, size=size),
                     0x3F800000 + rng.integers(0, 1 << 23, size=size))
        return torch.from_numpy(u.astype(np.int32)).cuda().view(F32)
    w = _f32_table(w, ones(1 << L, V))
    x = torch.zeros(B, N, device="cuda")
    at = torch.from_numpy(rng.integers(0, N, B)).cuda()
    x[torch.arange(B, device="cuda"), at] = ones(B)
    want = x.double() @ w.W.t()
    y = float(((w.linear(x).double() - want) / want).abs().max())
    dy = torch.zeros(B, M, device="cuda")
    at = torch.from_numpy(rng.integers(0, M, B)).cuda()
    dy[torch.arange(B, device="cuda"), at] = ones(B)
    want = dy.double() @ w.W
    dx = float(((w.backward(dy, dbias=False)[0].double() - want) / want).abs().max())
    _say(f"f32 single products M={M} N={N} B={B}: in units of 2^-23 {y * 2 ** 23:.3g} (y), "
         f"{dx * 2 ** 23:.3g} (dx), limit {lim * 2 ** 23:.3g}")
    assert max(y, dx) <= lim


@pytest.mark.parametrize("L,k,V,T,M,N,B", F32_SIZES)
def test_f32_keeps_all_bits(L, k, V, T, M, N, B):
    """Integers of 20 bits on either side of each product, three terms of 2 more bits to a
    sum: every product and sum is an fp32 number, so every output must be exact."""
    rng = np.random.default_rng(N)

    def sparse(rows, cols, values):
        t = torch.zeros(rows, cols, device="cuda")
        at = torch.from_numpy(rng.integers(0, cols, (rows, 3))).cuda()
        return t.scatter_(1, at, torch.from_numpy(values.astype(np.float32)).cuda())

    def wide(*size):
        return rng.integers(-(1 << 20) + 1, 1 << 20, size)

    def narrow(*size):
        return rng.choice([-4, -2, -1, 1, 2, 4], size)
    w = Coded(M + B, M, N, L, k, V, T, F32, False)
    for table, value in ((narrow, wide), (wide, narrow)):
        w = _f32_table(w, torch.from_numpy(table(1 << L, V).astype(np.float32)).cuda())
        x = sparse(B, N, value(B, 3))
        assert torch.equal(w.linear(x).double(), x.double() @ w.W.t())
        dy = sparse(B, M, value(B, 3))
        assert torch.equal(w.backward(dy, dbias=False)[0].double(), dy.double() @ w.W)
    # dw: three rows of the batch to each row of the matrix
    dy = sparse(M, B, wide(M, 3)).t().contiguous()
    xp = api.act_pack(torch.from_numpy(narrow(B, N).astype(np.float32)).cuda())
    _, dw, _ = w.backward(dy, dx=False, dbias=False, x=xp)
    xv = api.act_unpack(xp, F32).double()
    assert torch.equal(dw.double(), dy.double().t() @ xv)


@pytest.mark.parametrize("L,k,V,T,M,N,B", F32_SIZES)
def test_f32_rms(L, k, V, T, M, N, B):
    """N(0, 1) values: a random walk of K whole units 2^-23 over partial sums that grow like
    the root of their count is sqrt(K / 2) of them (halved: they are spread over a unit); two
    more for the products."""
    rng = np.random.default_rng(B)
    w = Coded(M + B, M, N, L, k, V, T, F32, False)

    def normal(*size):
        return torch.from_numpy(rng.standard_normal(size)).float().cuda()
    x, dy = normal(B, N), normal(B, M)
    xp = api.act_pack(x)
    xv = api.act_unpack(xp, F32).double()
    dx, dw, _ = w.backward(dy, x=xp)
    for name, got, want, K in (("y", w.linear(x), x.double() @ w.W.t(), N),
                               ("dx", dx, dy.double() @ w.W, M),
                               ("dw", dw, dy.double().t() @ xv, B)):
        rms = float((got.double() - want).square().mean().sqrt() / want.square().mean().sqrt())
        lim = (np.sqrt(K / 2) + 2) * 2.0 ** -24
        _say(f"f32 rms {name} M={M} N={N} B={B}: {rms:.3g}, limit {lim:.3g}")
        assert rms <= lim


def test_f32_near_the_largest_numbers():
    """Numbers whose first 16-bit term rounds past the largest: finite products, exact."""
    L, k, V, T, M, N, B = 16, 2, 1, 256, 130, 512, 300
    rng = np.random.default_rng(4)
    w = Coded(3, M, N, L, k, V, T, F32, False)
    w = _f32_table(w, torch.from_numpy(
        rng.choice([-0.5, -0.25, 0.25, 0.5], (1 << L, V)).astype(np.float32)).cuda())
    top = torch.finfo(F32).max
    x = torch.zeros(B, N, device="cuda")
    at = torch.from_numpy(rng.integers(0, N, B)).cuda()
    x[torch.arange(B, device="cuda"), at] = torch.from_numpy(
        rng.choice([top, -top, 0.999 * top, 0.998 * top], B).astype(np.float32)).cuda()
    assert torch.equal(w.linear(x).double(), x.double() @ w.W.t())
    dy = torch.zeros(B, M, device="cuda")
    dy[:, 5] = top
    assert torch.equal(w.backward(dy, dbias=False)[0].double(), dy.double() @ w.W)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("L,k,V,T,M,N,B", F32_SIZES + [(16, 2, 1, 256, 150, 512, 1),
                                                       (16, 2, 1, 256, 150, 512, 50)])
def test_rows_do_not_see_their_neighbours(L, k, V, T, M, N, B, dtype):
    """Bit for bit: an infinity, a NaN or the largest number in a row of x or dy changes that
    row's outputs (y, dx) alone, in a column of dy or a group of x that row or group of dw."""
    rng = np.random.default_rng(B + M)
    w = Coded(M + B, M, N, L, k, V, T, dtype, False)

    def normal(*size):
        return torch.from_numpy(rng.standard_normal(size)).to(dtype).cuda()
    a = torch.from_numpy(rng.standard_normal(M) / np.sqrt(N)).float().cuda()
    x, dy = normal(B, N), normal(B, M)

    def run(x, dy):
        dx, dw, _ = w.backward(dy, row_scale=a, x=api.act_pack(x))
        return w.linear(x, row_scale=a), dx, dw
    y, dx, dw = run(x, dy)
    for bad in (float("inf"), float("nan"), torch.finfo(dtype).max):
        row, col, out = B // 2, int(rng.integers(0, N)), int(rng.integers(0, M))
        xb, db = x.clone(), dy.clone()
        xb[row, col] = bad
        got = run(xb, dy)
        rows = torch.arange(B, device="cuda") != row
        cols = torch.arange(N, device="cuda") // 32 != col // 32
        _say(f"neighbours M={M} N={N} B={B} {dtype} {bad}")
        assert torch.equal(got[0][rows], y[rows]) and not torch.equal(got[0][row], y[row])
        assert torch.equal(got[1], dx) and torch.equal(got[2][:, cols], dw[:, cols])
        db[row, out] = bad
        got = run(x, db)
        keep = torch.arange(M, device="cuda") != out
        assert torch.equal(got[0], y) and torch.equal(got[1][rows], dx[rows])
        assert not torch.equal(got[1][row], dx[row])
        assert torch.equal(got[2][keep], dw[keep]) and not torch.equal(got[2][out], dw[out])


@pytest.mark.parametrize("B", [1, 40, 200])
def test_columns_of_one_buffer(B):
    """x, the residual, the output and guards as column ranges of one matrix; x itself as the
    output is refused."""
    M, N, dtype = 256, 256, BF16
    rng = np.random.default_rng(B)
    w = Coded(5, M, N, 16, 2, 1, 256, dtype, True)
    buf = torch.from_numpy(rng.integers(-8, 9, (B, 1024)).astype(np.float32)).to(dtype).cuda()
    x, out, res = buf[:, 8:264], buf[:, 264:520], buf[:, 520:776]
    keep = buf.clone()
    want = (x.double() @ w.W.t() + res.double()).to(dtype)
    w.linear(x, residual=res, out=out)
    assert torch.equal(out, want)
    out.copy_(keep[:, 264:520])
    assert torch.equal(buf, keep)
    for bad in (x, buf[:, 9:265], buf[:, 519:775]):
        with pytest.raises(_lib.TcqError) as e:
            w.linear(x, residual=res, out=bad)
        assert e.value.status == _lib.TCQ_EINVAL
    assert torch.equal(buf, keep)


def _terms_of_slope(z, act):
    """The two terms of act'(z), whose magnitudes bound its rounding."""
    if act == "silu":
        s = torch.sigmoid(z)
        return s, z * s * torch.sigmoid(-z)
    return 0.5 * torch.erfc(-z / np.sqrt(2.0)), z * torch.exp(-z * z / 2) / np.sqrt(2 * np.pi)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("B", [1, 20, 200])
def test_activations_keep_small_values(B, act, dtype):
    """act and its slope relative to their value, where it is far below |z| too: in fp32 to
    2^-20 (16 units; the formulas' roundings in fp32 arithmetic stay below 9), in 16-bit types
    to 2^-16 and the output's own rounding, from 2^-119 on.  z comes as the bias (x = 0) and
    as a checkpoint, dy is 1."""
    M, N = 6000, 256
    rng = np.random.default_rng(B)
    rel = 2.0 ** -20 if dtype == F32 else 2.0 ** -16
    for lo, hi in ((-8, -2), (-2, 2), (-14, 9), (-90, 90), (-1e4, 1e4)):
        w = Coded(3, M, N, 8, 2, 1, 64, dtype, True)
        z = torch.from_numpy(rng.uniform(lo, hi, M)).float().cuda()
        y = w.linear(torch.zeros(B, N, dtype=dtype, device="cuda"), bias=z, act=act)
        want = lc.act(z.double(), act)
        lim = rel * want.abs() + 2.0 ** -119
        lim = lim + lc.half(dtype) * (want.abs() + lim) + lc.tiny(dtype)
        r = float(((y.double() - want).abs() / lim).max())
        assert torch.equal(y, y[:1].expand(B, M))
        zp = api.act_pack(z.to(dtype).expand(B, M).contiguous())
        zv = api.act_unpack(zp, F32)[0].double()
        one = torch.zeros(B, M, dtype=dtype, device="cuda")
        one[B // 2] = 1
        db = w.backward(one, act=act, z=zp, dx=False)[2]
        first, second = _terms_of_slope(zv, act)
        lim = rel * (first.abs() + second.abs()) + 2.0 ** -119
        rs = float(((db.double() - first - second).abs() / lim).max())
        _say(f"small values B={B} {act} {dtype} [{lo}, {hi}]: worst error / bound {r:.3g}, "
             f"slope {rs:.3g}")
        assert max(r, rs) <= 1


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_activations_of_infinities(dtype):
    """z of +inf gives +inf, a NaN stays one, the largest finite numbers give themselves or 0."""
    M, N = 64, 256
    w = Coded(3, M, N, 8, 2, 1, 64, dtype, True)
    top = torch.finfo(dtype).max
    z = torch.zeros(M, device="cuda")
    z[:5] = torch.tensor([float("inf"), float("nan"), top, -top, float("-inf")])
    for act in ("silu", "gelu", "relu"):
        for B in (1, 200):
            y = w.linear(torch.zeros(B, N, dtype=dtype, device="cuda"), bias=z, act=act).float()
            assert bool((y[:, 0] == float("inf")).all()) and bool(torch.isnan(y[:, 1]).all())
            assert bool((y[:, 2] == top).all()) and bool((y[:, 3] == 0).all())
            assert bool((y[:, 5:] == 0).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_two_terms_of_one_number(act, dtype):
    """Products dy row_scale that fp32 rounds to the middle between two numbers of the type,
    from either side: the low term must belong to the high one that is stored.  A second row of
    the matrix takes the high term away (its row scale is 1), so dx is the low term."""
    rng = np.random.default_rng(13)
    bits = 12 if dtype == F16 else 9  # of a middle: one more than the type's
    dy, a = [], []
    for _ in range(40):
        v = torch.from_numpy(rng.uniform(1, 2, 1 << 17)).to(dtype).float().numpy()
        f = rng.uniform(0.25, 1, 1 << 17).astype(np.float32)
        exact = v.astype(np.float64) * f
        p = exact.astype(np.float32)
        m = np.frexp(p.astype(np.float64))[0] * 2.0 ** bits
        hit = (m == np.rint(m)) & (np.rint(m) % 2 == 1) & (exact != p)
        dy += list(v[hit][:8])
        a += list(f[hit][:8])
    R = len(dy)
    assert R > 50
    M, N = R + 1, 64
    w = Coded(1, M, N, 8, 2, 1, 64, dtype, False)
    w.table = torch.ones_like(w.table)
    scale = torch.ones(M, device="cuda")
    scale[:R] = torch.tensor(np.array(a), device="cuda")
    g = torch.zeros(R, M, dtype=dtype, device="cuda")
    v = torch.tensor(np.array(dy), device="cuda")
    at = torch.arange(R, device="cuda")
    s = v * scale[:R]
    high = s.to(dtype)
    g[at, at] = v.to(dtype)
    g[at, R] = -high
    z = api.act_pack(torch.ones(R, M, dtype=dtype, device="cuda"))
    dx = w.backward(g, row_scale=scale, act=act, z=z, dbias=False)[0]
    want = (v.double() * scale[:R].double() - high.double())[:, None].expand(R, N)
    lim = (4 * lc.U + lc.half(dtype) ** 2) * s.double().abs()[:, None]
    lim = lim + lc.half(dtype) * (want.abs() + lim) + lc.tiny(dtype)
    assert bool(((dx.double() - want).abs() <= lim).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_workspace_for_all_batches(dtype):
    """The workspace of the largest batch serves the smaller ones, whichever way they take."""
    M, N, most = 512, 1024, 2100
    rng = np.random.default_rng(1)
    w = Coded(5, M, N, 16, 2, 1, 256, dtype, True)
    x = torch.from_numpy(rng.integers(-8, 9, (most, N)).astype(np.float32)).to(dtype).cuda()
    dy = torch.from_numpy(rng.integers(-2, 3, (most, M)).astype(np.float32)).to(dtype).cuda()
    dt = api._DTYPES[dtype]
    ws = api.Workspace(_lib.tcq_decode_linear_workspace_bytes(dt, most, *w.shape))
    wb = api.Workspace(_lib.tcq_decode_linear_backward_workspace_bytes(dt, most, *w.shape, True,
                                                                       True, True))
    for B in (most, 1025, 520, 513, 512, 300, 129, 128, 40, 3, 1):
        y = w.linear(x[:B], workspace=ws)
        assert torch.equal(y, (x[:B].double() @ w.W.t()).to(dtype))
        xp = api.act_pack(x[:B])
        xv = api.act_unpack(xp, F32).double()
        dx, dw, db = w.backward(dy[:B], x=xp, workspace=wb)
        g = dy[:B].double()
        assert torch.equal(dx, (g @ w.W).to(dtype)) and torch.equal(dw, (g.t() @ xv).to(dtype))
        assert torch.equal(db.double(), g.sum(0))


def test_workspace_of_another_device():
    """A workspace in host memory is refused before the call."""
    w = Coded(5, 64, 512, 16, 2, 1, 256, F16, True)
    x = torch.ones(300, 512, dtype=F16, device="cuda")
    dy = torch.ones(300, 64, dtype=F16, device="cuda")
    ws = api.Workspace(1 << 24, "cpu")
    with pytest.raises(AssertionError, match="workspace"):
        w.linear(x, workspace=ws)
    with pytest.raises(AssertionError, match="workspace"):
        w.backward(dy, workspace=ws)
    ws = api.Workspace(1 << 24)
    assert torch.equal(w.linear(x, workspace=ws), w.linear(x))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gradients_of_spread_row_scales(dtype):
    """Row scales over 24 powers of two in one matrix."""
    M, N, B = 300, 512, 60
    rng = np.random.default_rng(21)
    w = Coded(6, M, N, 16, 2, 1, 256, dtype, False)

    def normal(*size):
        return torch.from_numpy(rng.standard_normal(size)).to(dtype).cuda()
    a = torch.from_numpy(rng.standard_normal(M) * 2.0 ** rng.integers(-18, 7, M)).float().cuda()
    r = _gradients(w, normal(B, M), a, "gelu", normal(B, M), normal(B, N), dtype)
    _say(f"spread row scales {dtype}: worst error / bound dx {r[0]:.3g}, dw {r[1]:.3g}")
    assert max(r) <= 1


@pytest.mark.parametrize("B", [5, 300])
def test_row_scale_changes_between_replays(B):
    """fp16 gradients in a captured graph: the power of two comes from the row scale of the
    moment, and every replay equals the eager call."""
    M, N, dtype = 384, 512, F16
    w = Coded(4, M, N, 16, 2, 1, 256, dtype, False)
    g = torch.Generator("cuda").manual_seed(B)

    def normal(*size):
        return torch.randn(*size, generator=g, device="cuda")
    dy, a = normal(B, M).to(dtype), normal(M)
    zp, xp = api.act_pack(normal(B, M).to(dtype)), api.act_pack(normal(B, N).to(dtype))

    def step():
        return w.backward(dy, row_scale=a, act="silu", z=zp, x=xp)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for size in (2.0 ** -12, 1.0, 3000.0, 2.0 ** -5):
        a.copy_(normal(M) * size)
        dy.copy_(normal(B, M) / max(size, 1.0))
        want = step()
        torch.cuda.synchronize()
        assert bool(torch.isfinite(want[0]).all())
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(outs, want):
            assert torch.equal(p, q), size
