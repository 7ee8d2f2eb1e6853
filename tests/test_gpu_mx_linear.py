"""The microscaled linear layer and its gradients against float64 forms, within bounds counted
from the kernels' roundings (mx_check), and bit for bit where every sum is exact."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import api  # noqa: E402

import mx_check as mc  # noqa: E402
from linear_check import U, half, tiny  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]
FORMATS = ["fp4", "fp8"]
NAN = float("nan")


def _say(msg):
    sys.stdout.write(msg + "\n")
    sys.stdout.flush()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _weights(g, M, N):
    return api.mx_pack(_randn(g, M, N) * torch.exp(0.5 * _randn(g, M, 1)) / max(N, 1) ** 0.5,
                       "fp4")


def _values(p):
    return api.mx_unpack(p, torch.float32).double()


def _inside(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), \
        f"{what}: {int(bad.sum())} outside, worst {float((off / bound).max()):.3g} of the bound"


# few rows (quantised in the kernel or before it, in one share or several), 128 x 128 tiles whole
# and split, 256 x 256 ones
SIZES = [(513, 17, 96), (600, 70, 2100), (1000, 1100, 700), (1100, 2050, 520), (1, 1, 1), (1, 16, 32), (2, 17, 33), (5, 100, 130), (16, 48, 1000), (17, 64, 256),
         (33, 40, 515), (70, 130, 129), (128, 200, 544), (129, 130, 260), (300, 513, 1100),
         (1030, 2050, 200), (200, 144, 4096), (2049, 4000, 96), (3, 2000, 9000),
         (130, 7300, 6190), (1150, 1700, 6300)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,M,N", SIZES)
def test_linear(B, M, N, dtype, fmt):
    _say(f"linear {B}x{M}x{N} {dtype} {fmt}")
    g = _gen(B + M + N)
    w = _weights(g, M, N)
    x = (_randn(g, B, N) * torch.exp(0.5 * _randn(g, 1, N))).to(dtype)
    bias = _randn(g, M) if B % 2 else None
    res = _randn(g, B, M).to(dtype) if M % 2 == 0 else None
    xq = mc.quantised(x, fmt)
    want, mag = mc.linear(xq, _values(w), bias, res)
    bound = mc.linear_bound(want, mag, bias, res, N, dtype)
    y = api.mx_linear(x, w, bias=bias, residual=res, x_format=fmt)
    _inside(y, want, bound, "dense x")
    y2, kept = api.mx_linear(x, w, bias=bias, residual=res, x_format=fmt, keep=True)
    p = api.mx_pack(x, fmt)
    assert torch.equal(kept.codes, p.codes) and torch.equal(kept.scale, p.scale)
    y3 = api.mx_linear(p, w, bias=bias, residual=res, dtype=dtype)
    _inside(y2, want, bound, "codes kept")
    # the way to the product does not change it
    assert torch.equal(y, y2) and torch.equal(y, y3)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B,M,N", SIZES)
def test_exact_sums(B, M, N, fmt):
    """Inputs on a grid on which every partial sum is an fp32 number: equal bit for bit."""
    g = _gen(B * 3 + M + N)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")

    def draw(rows, cols):
        v = grid[torch.randint(0, 8, (rows, cols), generator=g, device="cuda")]
        v = v * torch.where(torch.rand(rows, cols, generator=g, device="cuda") < 0.5, -1.0, 1.0)
        v[:, ::32] = 4.0  # every group's scale is its power of two below
        e = torch.randint(-1, 2, (rows, -(-cols // 32)), generator=g, device="cuda").float()
        return v * torch.exp2(e).repeat_interleave(32, 1)[:, :cols]

    xv, wv = draw(B, N), draw(M, N)
    # fp8 holds the same values: two mantissa bits, three binades
    y = api.mx_linear(xv, api.mx_pack(wv, "fp4"), x_format=fmt)
    assert torch.equal(y.double(), xv.double() @ wv.double().t().contiguous())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B", [1, 9, 40, 150, 1000, 6700])
def test_scales_meet_their_groups(B, fmt):
    """One non-zero group of x at a time, every scale different: a scale that is read for another
    group, row or operand changes the result."""
    M, N = 272, 1088
    g = _gen(B)
    wv = torch.ones(M, N, device="cuda") * torch.exp2(
        torch.randint(-30, 30, (M, N // 32), generator=g, device="cuda").float()
    ).repeat_interleave(32, 1)
    x = torch.zeros(B, N, device="cuda")
    group = torch.randint(0, N // 32, (B,), generator=g, device="cuda")
    e = torch.exp2(torch.randint(-30, 30, (B,), generator=g, device="cuda").float())
    for b in range(B):
        x[b, group[b] * 32:group[b] * 32 + 32] = e[b]
    y = api.mx_linear(x, api.mx_pack(wv, "fp4"), x_format=fmt)
    want = 32 * e.double()[:, None] * wv.double()[:, ::32].t()[group]
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B", [1, 20, 200, 7300])
def test_nan_stays_in_its_row(B, dtype, fmt):
    M, N = 520, 256
    g = _gen(B)
    w = _weights(g, M, N)
    x = _randn(g, B, N).to(dtype)
    clean = api.mx_linear(x, w, x_format=fmt)
    x[B // 2, 100] = NAN
    w.scale[7, 3] = 255
    y = api.mx_linear(x, w, x_format=fmt)
    bad = torch.zeros(B, M, dtype=torch.bool, device="cuda")
    bad[B // 2], bad[:, 7] = True, True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B", [3, 60, 400])
def test_strided_and_in_place(B, fmt):
    """Rows of wider matrices that start anywhere, y over the residual, guard columns kept."""
    M, N, dtype = 77, 200, torch.bfloat16
    g = _gen(B)
    big = api.mx_pack(_randn(g, M, N + 96), "fp4")
    w = api.MxPacked(big.codes[:, 16:16 + 7 * 16], big.scale[:, 1:8].contiguous(), 7 * 32, "fp4")
    N = w.cols
    xw = torch.full((B, N + 9), NAN, dtype=dtype, device="cuda")
    xw[:, 3:3 + N] = _randn(g, B, N).to(dtype)
    x = xw[:, 3:3 + N]
    out = torch.full((B + 1, M + 5), 3.0, dtype=dtype, device="cuda")
    out[:B, 1:1 + M] = _randn(g, B, M).to(dtype)
    res = out[:B, 1:1 + M].clone()
    want, mag = mc.linear(mc.quantised(x, fmt), _values(
        api.MxPacked(w.codes.contiguous(), w.scale, N, "fp4")), None, res)
    y = api.mx_linear(x, w, residual=out[:B, 1:1 + M], out=out[:B, 1:1 + M], x_format=fmt)
    _inside(y, want, mc.linear_bound(want, mag, None, res, N, dtype), "in place")
    assert bool((out[:, 0] == 3).all()) and bool((out[:, 1 + M:] == 3).all())
    assert bool((out[B] == 3).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_workspace_for_smaller_batches(fmt):
    M, N = 300, 640
    g = _gen(1)
    w = _weights(g, M, N)
    from trellis_coded_bit_amd import _lib
    sizes = [_lib.tcq_mx_linear_workspace_bytes(api._FORMATS[fmt], B, M, N)
             for B in (1, 16, 17, 128, 129, 200, 255, 256, 257, 512, 513, 1000, 5000,
                       7000)]
    assert sizes == sorted(sizes)
    ws = api.Workspace(sizes[-1])
    for B in (7000, 1, 129, 40, 600):
        x = _randn(g, B, N).bfloat16()
        assert torch.equal(api.mx_linear(x, w, x_format=fmt, workspace=ws),
                           api.mx_linear(x, w, x_format=fmt))


def test_empty_sizes():
    g = _gen(2)
    bias = _randn(g, 50)
    for fmt in FORMATS:
        for B in (1, 200, 3000):
            w = api.mx_pack(torch.zeros(50, 0, device="cuda"), "fp4")
            x = torch.zeros(B, 0, device="cuda")
            assert torch.equal(api.mx_linear(x, w, bias=bias, x_format=fmt),
                               bias.expand(B, 50))
        w = _weights(g, 50, 64)
        assert api.mx_linear(torch.zeros(0, 64, device="cuda"), w, x_format=fmt).shape == (0, 50)
        w = api.mx_pack(torch.zeros(0, 64, device="cuda"), "fp4")
        assert api.mx_linear(torch.zeros(5, 64, device="cuda"), w, x_format=fmt).shape == (5, 0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B", [1, 50, 300, 7200])
def test_streams_and_graph(B, fmt):
    M, N = 256, 1024
    g = _gen(3)
    w = _weights(g, M, N)
    x = _randn(g, B, N).bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = api.mx_linear(x, w, x_format=fmt)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, api.mx_linear(x, w, x_format=fmt))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, kept = api.mx_linear(x, w, x_format=fmt, keep=True)
        dx, dw, db = api.mx_linear_backward(y, w, kept)
    for _ in range(3):
        x.copy_(_randn(g, B, N).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        y2, kept2 = api.mx_linear(x, w, x_format=fmt, keep=True)
        assert torch.equal(y, y2) and torch.equal(kept.codes, kept2.codes)
        for a, b in zip((dx, dw, db), api.mx_linear_backward(y2, w, kept2)):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- gradients

GRAD_SIZES = [(1, 1, 1), (3, 17, 33), (5, 8, 130), (64, 100, 1000), (200, 257, 96),
              (300, 512, 520), (1000, 72, 2048)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,M,N", GRAD_SIZES)
def test_gradients(B, M, N, dtype, fmt):
    _say(f"gradients {B}x{M}x{N} {dtype} {fmt}")
    g = _gen(B + 2 * M + N)
    w = _weights(g, M, N)
    x = api.mx_pack(_randn(g, B, N), fmt)
    dy = _randn(g, B, M).to(dtype)
    dx, dw, db = api.mx_linear_backward(dy, w, x)
    W, X, d = _values(w), _values(x), dy.double()

    def check(got, a, b, K, what):
        want, mag = a @ b, a.abs() @ b.abs()
        e = mc.gamma(K, dtype) * mag
        # products of fp32 terms leave out less than 2^-22 of each
        e = e + (2.0 ** -22 * mag if dtype == torch.float32 else 0)
        _inside(got, want, e + half(dtype) * (want.abs() + e) + tiny(dtype), what)

    check(dx, d, W, M, "dx")
    check(dw, d.t().contiguous(), X, B, "dw")
    want = d.sum(0)
    _inside(db, want, 2 * (B + 1) * U * d.abs().sum(0) + tiny(torch.float32), "dbias")
    # parts of the call
    assert torch.equal(api.mx_linear_backward(dy, w, None, dbias=False)[0], dx)
    _, dw2, db2 = api.mx_linear_backward(dy, w, x, dx=False)
    assert torch.equal(dw2, dw) and torch.equal(db2, db)


@pytest.mark.parametrize("scale", [2.0 ** -30, 2.0 ** 20])
def test_fp16_gradients_of_far_scales(scale):
    """Weights and inputs that fp16 holds with few bits or not at all."""
    B, M, N = 40, 64, 96
    g = _gen(9)
    w = api.mx_pack(_randn(g, M, N) * scale, "fp4")
    x = api.mx_pack(_randn(g, B, N) * scale, "fp8")
    # (tiny weights: the gradients fall among fp16's subnormals, whose spacing the bound counts)
    dy = (_randn(g, B, M) * (2.0 ** -14 if scale > 1 else 1000.0)).to(torch.float16)
    dx, dw, _ = api.mx_linear_backward(dy, w, x)
    for got, a, b, K in ((dx, dy.double(), _values(w), M),
                         (dw, dy.double().t().contiguous(), _values(x), B)):
        want, mag = a @ b, a.abs() @ b.abs()
        e = mc.gamma(K) * mag
        _inside(got, want, e + half(torch.float16) * (want.abs() + e) + tiny(torch.float16),
                f"scale {scale}")


def test_gradients_are_differences():
    """y is linear in W's and x's values: differences of calls on values the formats hold exactly."""
    B, M, N = 6, 40, 64
    g = _gen(10)
    grid = torch.tensor([0.0, 1.0, 2.0, 4.0, -1.0, -2.0, -4.0], device="cuda")

    def draw(rows):
        v = grid[torch.randint(0, 7, (rows, N), generator=g, device="cuda")]
        v[:, ::32] = 4.0
        return v

    xv, wv = draw(B), draw(M)
    w, dy = api.mx_pack(wv, "fp4"), _randn(g, B, M)
    _, kept = api.mx_linear(xv, w, x_format="fp4", keep=True)
    dx, dw, db = api.mx_linear_backward(dy, w, kept)

    def loss(x, w, bias=None):
        return (api.mx_linear(x, api.mx_pack(w, "fp4"), bias=bias, x_format="fp4").double()
                * dy.double()).sum()

    for i, j in ((0, 1), (3, 40), (5, 63)):
        a, b = xv.clone(), xv.clone()
        a[i, j], b[i, j] = 3.0, -1.0
        d = float(loss(a, wv) - loss(b, wv)) / 4
        assert abs(d - float(dx[i, j])) <= 2.0 ** -16 * float(dy.abs().sum() * 8)
        a, b = wv.clone(), wv.clone()
        a[i, j], b[i, j] = 3.0, -1.0
        d = float(loss(xv, a) - loss(xv, b)) / 4
        assert abs(d - float(dw[i, j])) <= 2.0 ** -16 * float(dy.abs().sum() * 8)
    bias = torch.zeros(M, device="cuda")
    bias[3] = 1.0
    d = float(loss(xv, wv, bias) - loss(xv, wv))
    assert abs(d - float(db[3])) <= 2.0 ** -16 * float(dy.abs().sum() * 64)


@pytest.mark.parametrize("dtype", TYPES)
def test_gradients_of_nothing(dtype):
    g = _gen(11)
    w = _weights(g, 40, 64)
    x = api.mx_pack(torch.zeros(0, 64, device="cuda"), "fp8")
    dx, dw, db = api.mx_linear_backward(torch.zeros(0, 40, device="cuda", dtype=dtype), w, x)
    assert dx.shape == (0, 64) and float(dw.abs().max()) == 0 and float(db.abs().max()) == 0
    w = api.mx_pack(torch.zeros(0, 64, device="cuda"), "fp4")
    dx, dw, db = api.mx_linear_backward(torch.zeros(7, 0, device="cuda", dtype=dtype), w)
    assert float(dx.abs().max()) == 0


def test_strided_dy():
    """dy whose rows start anywhere, and one that the products read where it lies: the same."""
    B, M, N = 90, 64, 128
    g = _gen(12)
    w, x = _weights(g, M, N), api.mx_pack(_randn(g, B, N), "fp4")
    for dtype in TYPES:
        dy = _randn(g, B, M).to(dtype)
        wide = torch.full((B, M + 7), NAN, dtype=dtype, device="cuda")
        wide[:, 3:3 + M] = dy
        for a, b in zip(api.mx_linear_backward(dy, w, x),
                        api.mx_linear_backward(wide[:, 3:3 + M], w, x)):
            assert torch.equal(a, b)
