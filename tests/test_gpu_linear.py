"""The coded linear layer (tcq_decode_linear) and its gradients (tcq_decode_linear_backward)
against the oracle's decode followed by float64 products.

Bars (see linear_check.py): on exact inputs (codebook on a 1/8 grid, small-integer x, scales
that are powers of two) every product and sum is an fp32 number in any order, so each output
must equal the reference rounded once; on N(0, 1) inputs each output must lie within a
bound that counts the roundings.
"""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import _lib, api  # noqa: E402
from trellis_coded_bit_amd import workloads as wl  # noqa: E402

import linear_check as lc  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]
ACTS = ["none", "relu", "silu", "gelu"]


def _say(msg):
    sys.stdout.write(msg + "\n")
    sys.stdout.flush()


class Coded:
    """A coded matrix on the GPU and its float64 values."""

    def __init__(self, seed, M, N, L, k, V, T, dtype, exact, oracle=None, shift=0):
        rng = np.random.default_rng(seed)
        self.shape = (M, N, L, k, V, T)
        bits, s0 = lc.random_streams(rng, M * (N // T), L, k, V, T)
        if exact:
            C = lc.grid_table(L, V, rng)
        else:
            C = rng.standard_normal((1 << L, V)).astype(np.float32)
        table = torch.from_numpy(C).to(dtype)
        flat = torch.zeros(table.numel() + shift, dtype=dtype)
        flat[shift:] = table.reshape(-1)
        self.table = flat.cuda()[shift:].view(table.shape)
        self.bits = torch.from_numpy(bits.view(np.int32)).cuda()
        self.s0 = torch.from_numpy(s0.view(np.int32)).cuda()
        rounded = np.ascontiguousarray(table.float().numpy())
        if oracle is not None:
            W = torch.from_numpy(oracle.decode_matrix(bits, s0, rounded, M, N, L, k, V, T)).cuda()
        else:  # the library's decode, which has tests of its own, bit for bit
            W = api.decode(self.bits, self.s0, torch.from_numpy(rounded).cuda(), M, N, L, k, V, T)
        self.W = W.double()

    def linear(self, x, **kw):
        return api.decode_linear(self.bits, self.s0, self.table, x, *self.shape, **kw)

    def backward(self, dy, **kw):
        return api.decode_linear_backward(self.bits, self.s0, self.table, dy, *self.shape, **kw)


def _place(t, lead, first, fill=float("nan")):
    """t as a column slice of a wider GPU matrix whose other columns are `fill`."""
    wide = torch.full((t.shape[0] + 1, t.shape[1] + lead), fill, dtype=t.dtype, device="cuda")
    view = wide[:t.shape[0], first:first + t.shape[1]]
    view.copy_(t)
    return view


def _ints(rng, rows, cols, dtype, most=8):
    return torch.from_numpy(rng.integers(-most, most + 1, size=(rows, cols)).astype(np.float32)
                            ).to(dtype).cuda()


# L, k, V, T, M, N: whole units and not, one to four values a step, odd sizes
SHAPES = [
    (16, 2, 1, 256, 130, 512), (16, 2, 2, 256, 33, 256), (16, 3, 1, 256, 70, 768),
    (8, 2, 1, 64, 64, 64), (12, 2, 1, 64, 257, 192), (16, 4, 1, 256, 40, 256),
    (10, 3, 2, 30, 21, 120), (16, 1, 1, 17, 19, 17 * 7), (4, 1, 1, 12, 5, 36),
    (16, 2, 4, 64, 48, 128), (9, 4, 1, 100, 6, 300), (16, 3, 1, 1, 9, 5),
]


def _exact_forward(w, x, rng, dtype, act, residual, strided, bias=True):
    M = w.shape[0]
    B = x.shape[0]
    a = torch.from_numpy(2.0 ** rng.integers(-1, 2, M)).float().cuda()
    b = torch.from_numpy(rng.integers(-64, 65, M) / 16.0).float().cuda() if bias else None
    res = _ints(rng, B, M, dtype) if residual else None
    if strided and res is not None:
        res = _place(res, 5, 2)
    z, y, _ = lc.forward(w.W, x.double(), a.double(), None if b is None else b.double(), act,
                         None if res is None else res.double())
    got, pre = w.linear(x, row_scale=a, bias=b, act=act, residual=res, pre=True)
    torch.cuda.synchronize()
    assert torch.equal(pre, z.to(dtype))
    assert torch.equal(got, y.to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_exact(oracle_lib, shape, dtype):
    import oracle
    L, k, V, T, M, N = shape
    rng = np.random.default_rng(M * 31 + N)
    w = Coded(M + N, M, N, L, k, V, T, dtype, True, oracle)
    for B in (1, 2, 7, 16, 33, 100, 129):
        _say(f"linear exact {shape} {dtype} B={B}")
        for strided in (False, True):
            x = _ints(rng, B, N, dtype)
            x = _place(x, 9, 3) if strided else x
            _exact_forward(w, x, rng, dtype, "relu" if B % 2 else "none", strided, strided)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(2, 1, 1, 32, 9, 96), (3, 2, 1, 32, 17, 64),
                                   (3, 1, 2, 64, 20, 64), (5, 1, 1, 160, 33, 160),
                                   (16, 2, 1, 32, 18, 4096 + 32), (14, 2, 2, 96, 40, 96 * 7)])
def test_linear_exact_small_tables_and_blocks(oracle_lib, shape, dtype):
    """Tables of a few bytes, blocks of one run of 32 columns, rows that are no whole unit
    of columns, and a codebook that does not start on 16 bytes."""
    import oracle
    L, k, V, T, M, N = shape
    rng = np.random.default_rng(L + N)
    for shift in (0, 1):
        w = Coded(L + N, M, N, L, k, V, T, dtype, True, oracle, shift)
        for B in (1, 16, 17, 40, 70, 128, 150):
            _say(f"linear small tables {shape} {dtype} B={B} shift={shift}")
            _exact_forward(w, _ints(rng, B, N, dtype), rng, dtype, "none", True, False)
        dy, xp = _ints(rng, 20, M, dtype, 4), api.act_pack(_ints(rng, 20, N, dtype))
        dx, dw, _ = w.backward(dy, x=xp)
        assert torch.equal(dx, (dy.double() @ w.W).to(dtype))
        xv = api.act_unpack(xp, torch.float32).double()
        assert torch.equal(dw, (dy.double().t() @ xv).to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,k,V,T", [(16, 2, 1, 256), (16, 2, 2, 256), (12, 2, 1, 64)])
def test_linear_infinities_stay_infinities(L, k, V, T, dtype):
    """An infinity in x meets every weight of its column once: with no zero in the table
    the outputs of that row are infinities of the weight's sign, not NaN, whichever part of
    the table the weight lies in."""
    M, N = 80, 512
    w = Coded(L + V, M, N, L, k, V, T, dtype, True)
    w.table[w.table == 0] = 1.0
    W = api.decode(w.bits, w.s0, w.table.float(), M, N, L, k, V, T).double()
    for B in (1, 20, 100, 300):
        x = torch.ones(B, N, dtype=dtype, device="cuda")
        x[B // 2, N // 3] = float("inf")
        y = w.linear(x)
        want = (torch.ones(B, N, device="cuda", dtype=torch.float64) @ W.t()).to(dtype)
        want[B // 2] = torch.sign(W[:, N // 3]).to(dtype) * float("inf")
        assert torch.equal(y, want)


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -60, 1.0, 2.0 ** 60, 2.0 ** 100])
def test_linear_f32_magnitudes(scale):
    """fp32 over the type's range: the bound of six bf16 products each, and a relative rms
    error of a few fp32 units, as a sum of fp32 products has."""
    M, N, B = 130, 1024, 300
    rng = np.random.default_rng(2)
    w = Coded(17, M, N, 16, 2, 1, 256, torch.float32, False)
    x = torch.from_numpy(rng.standard_normal((B, N)) * scale).float().cuda()
    y = w.linear(x)
    want = x.double() @ w.W.t()
    mag = x.double().abs() @ w.W.abs().t()
    lim = lc.gamma(N, torch.float32) * mag
    ratio = float(((y.double() - want).abs() / lim).max())
    rms = float((y.double() - want).square().mean().sqrt() / want.square().mean().sqrt())
    _say(f"  f32 scale {scale:.3g}: worst error / bound {ratio:.3g}, relative rms {rms:.3g}")
    assert ratio <= 1 and rms < 1e-6
    dy = torch.from_numpy(rng.standard_normal((B, M)) * scale).float().cuda()
    dx, _, _ = w.backward(dy, dbias=False)
    want, mag = dy.double() @ w.W, dy.double().abs() @ w.W.abs()
    assert bool(((dx.double() - want).abs() <= lc.gamma(M, torch.float32) * mag).all())


def test_linear_f32_below_the_terms():
    """Numbers whose smallest term falls below bf16's smallest: within 2^-133 each."""
    M, N, B = 130, 256, 300
    rng = np.random.default_rng(2)
    w = Coded(18, M, N, 16, 2, 1, 256, torch.float32, False)
    x = torch.from_numpy(rng.standard_normal((B, N)) * 2.0 ** -116).float().cuda()
    y = w.linear(x)
    want = x.double() @ w.W.t()
    lim = lc.gamma(N, torch.float32) * (x.double().abs() @ w.W.abs().t())
    lim = lim + 2.0 ** -133 * w.W.abs().sum(1) + lc.tiny(torch.float32) * 6 * N
    ratio = float(((y.double() - want).abs() / lim).max())
    _say(f"  f32 tiny: worst error / bound {ratio:.3g}")
    assert ratio <= 1


@pytest.mark.parametrize("L,k,V,T,M,N,B", [
    (8, 2, 1, 32, 32768, 32, 70000),       # more than 2^31 outputs
    (8, 2, 1, 32, 64, 32, 1),              # and the smallest
])
def test_linear_offsets_past_32_bits(L, k, V, T, M, N, B):
    _say(f"linear many outputs B={B} M={M}")
    dtype = torch.bfloat16
    rng = np.random.default_rng(1)
    w = Coded(9, M, N, L, k, V, T, dtype, True)
    x = _ints(rng, B, N, dtype)
    y, z = w.linear(x, act="relu", pre=True)
    rows = torch.unique(torch.tensor([0, B // 2, B - 1], device="cuda"))
    want = x[rows].double() @ w.W.t()
    assert torch.equal(z[rows], want.to(dtype))
    assert torch.equal(y[rows], want.clamp_min(0).to(dtype))
    dy = torch.zeros_like(y)
    dy[rows] = _ints(rng, rows.numel(), M, dtype, 4)
    xp = api.act_pack(x)
    dx, dw, db = w.backward(dy, act="relu", z=api.act_pack(z), x=xp)
    zp = api.act_pack(z[rows].contiguous())
    g = dy[rows].double() * (api.act_unpack(zp, torch.float32) > 0)
    assert torch.equal(dx[rows], (g @ w.W).to(dtype))
    assert torch.equal(db.double(), g.sum(0))
    xv = api.act_unpack(xp, torch.float32).double()
    assert torch.equal(dw, (g.t() @ xv[rows]).to(dtype))


def test_linear_far_apart_rows():
    """A leading dimension above 2^21 values, and rows that start on odd addresses."""
    dtype = torch.bfloat16
    M, N, B = 96, 512, 140
    w = Coded(11, M, N, 16, 2, 1, 256, dtype, True)
    ld = (1 << 21) + 24
    buf = torch.zeros(B * ld, dtype=dtype, device="cuda")
    for first in (0, 3):
        x = buf[first:].as_strided((B, N), (ld, 1))
        x.copy_(_ints(np.random.default_rng(first), B, N, dtype))
        for rows in (1, 16, 50, B):
            y = w.linear(x[:rows])
            assert torch.equal(y, (x[:rows].double() @ w.W.t()).to(dtype))


def test_threads_on_own_streams():
    """Four host threads, each on its own stream, forward and backward at once: the bits of
    the same calls made one after another."""
    import threading
    dtype = torch.bfloat16
    M, N = 256, 1024
    w = Coded(6, M, N, 16, 2, 1, 256, dtype, False)
    g = torch.Generator("cuda").manual_seed(3)
    inputs = [(torch.randn(B, N, generator=g, device="cuda").to(dtype),
               torch.randn(B, M, generator=g, device="cuda").to(dtype)) for B in (1, 30, 90, 400)]

    def step(x, dy):
        y, z = w.linear(x, act="silu", pre=True)
        return [y, *w.backward(dy, act="silu", z=api.act_pack(z), x=api.act_pack(x))]
    want = [step(*p) for p in inputs]
    torch.cuda.synchronize()
    got, errs = [None] * 4, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(5):
                    got[i] = step(*inputs[i])
                s.synchronize()
        except Exception as e:  # reported below
            errs.append(e)
    ths = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in ths:
        t.start()
    for t in ths:
        t.join(timeout=60)
    assert not any(t.is_alive() for t in ths) and not errs, errs
    for p, q in zip(want, got):
        for u, v in zip(p, q):
            assert torch.equal(u, v)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,k,V,T,M,N,B", [
    (16, 2, 1, 256, 2048, 2048, 1), (16, 2, 2, 256, 14336, 4096, 3),
    (16, 3, 1, 256, 4096, 14336, 17), (16, 2, 1, 256, 4096, 4096, 500),
    (16, 2, 1, 256, 4100, 4096, 2049), (12, 2, 1, 64, 1031, 4160, 1027)])
def test_linear_exact_large(L, k, V, T, M, N, B, dtype):
    _say(f"linear exact large L={L} k={k} V={V} M={M} N={N} B={B} {dtype}")
    rng = np.random.default_rng(B)
    w = Coded(B, M, N, L, k, V, T, dtype, True)
    _exact_forward(w, _ints(rng, B, N, dtype), rng, dtype, "none", True, False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape,B", [(SHAPES[0], 5), (SHAPES[1], 64), (SHAPES[2], 200),
                                     (SHAPES[6], 3)])
def test_linear_within_bounds(oracle_lib, shape, B, act, dtype):
    import oracle
    L, k, V, T, M, N = shape
    _say(f"linear bounds {shape} B={B} {act} {dtype}")
    rng = np.random.default_rng(N + B)
    w = Coded(N, M, N, L, k, V, T, dtype, False, oracle)

    def normal(*size):
        return torch.from_numpy(rng.standard_normal(size)).to(dtype).cuda()
    x, res = normal(B, N), normal(B, M)
    a = torch.from_numpy(rng.standard_normal(M) / np.sqrt(N)).float().cuda()
    b = torch.from_numpy(rng.standard_normal(M)).float().cuda()
    y, z = w.linear(x, row_scale=a, bias=b, act=act, residual=res, pre=True)
    torch.cuda.synchronize()
    ez, ey, mag = lc.forward(w.W, x.double(), a.double(), b.double(), act, res.double())
    dz, dy = lc.forward_bounds(ez, ey, mag, res, act, N, dtype)
    rz, ry = float(((z.double() - ez).abs() / dz).max()), float(((y.double() - ey).abs() / dy).max())
    _say(f"  worst error / bound: z {rz:.3g}, y {ry:.3g}")
    assert rz <= 1 and ry <= 1


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B", [1, 5, 40, 300])
def test_linear_rows_are_their_own(dtype, B):
    """A NaN or an infinity in a row of x reaches that row alone, padding is not read, and
    nothing outside the output is written; in place of the residual too."""
    L, k, V, T, M, N = 16, 2, 1, 256, 150, 512
    _say(f"linear rows {dtype} B={B}")
    rng = np.random.default_rng(B)
    w = Coded(B, M, N, L, k, V, T, dtype, True)
    x = _place(_ints(rng, B, N, dtype), 8, 0)
    want = (x.double() @ w.W.t())
    bad = B // 2
    x[bad, N - 1] = float("inf") if B % 2 else float("nan")
    buf = torch.full((B + 2, M + 6), 7.0, dtype=dtype, device="cuda")
    out = buf[1:B + 1, 2:M + 2]
    res = _ints(rng, B, M, dtype)
    out.copy_(res)
    y = w.linear(x, residual=out, out=out)
    torch.cuda.synchronize()
    assert y.data_ptr() == out.data_ptr()
    keep = torch.arange(B, device="cuda") != bad
    assert torch.equal(y[keep], (want + res.double())[keep].to(dtype))
    col = w.W[:, N - 1]
    hit = y[bad][col != 0]
    assert not bool(torch.isfinite(hit).any())
    buf[1:B + 1, 2:M + 2] = 7.0
    assert bool((buf == 7.0).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_linear_empty(dtype):
    C = torch.zeros(1 << 16, 1, dtype=dtype, device="cuda")
    for M, N, B in [(3, 0, 4), (3, 512, 0), (0, 512, 4), (0, 0, 0)]:
        nb = M * (N // 256)
        bits = torch.zeros(nb, 16, dtype=torch.int32, device="cuda")
        s0 = torch.zeros(nb, dtype=torch.int32, device="cuda")
        b = torch.arange(M, device="cuda", dtype=torch.float32)
        x = torch.ones(B, N, dtype=dtype, device="cuda")
        y = api.decode_linear(bits, s0, C, x, M, N, 16, 2, 1, 256, bias=b)
        assert y.shape == (B, M)
        if M and B and N == 0:
            assert torch.equal(y, b.to(dtype).expand(B, M))
        p = api.act_pack(x)
        dx, dw, db = api.decode_linear_backward(bits, s0, C, torch.ones(B, M, dtype=dtype,
                                                                        device="cuda"), M, N,
                                                16, 2, 1, 256, x=p)
        assert dx.shape == (B, N) and dw.shape == (M, N)
        assert torch.equal(dx, torch.zeros_like(dx)) and torch.equal(db, torch.full_like(db, B))
        if B == 0:
            assert torch.equal(dw, torch.zeros_like(dw))


def _grad_reference(w, dy, a, act, z, x, dtype, rounded):
    """float64 gradients from the checkpoints' values; s rounded to the layer's type when
    `rounded`."""
    g = dy.double()
    if act != "none":
        g = g * lc.slope(z, act)
    s = g if a is None else g * a.double()
    if rounded:
        s = s.to(dtype).double()
    return g, s, s @ w.W, s.t() @ x


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_backward_exact(oracle_lib, shape, dtype):
    import oracle
    L, k, V, T, M, N = shape
    rng = np.random.default_rng(M * 17 + N)
    w = Coded(M * 3 + N, M, N, L, k, V, T, dtype, True, oracle)
    for B, act in [(1, "none"), (2, "relu"), (19, "relu"), (64, "none"), (131, "relu")]:
        _say(f"backward exact {shape} {dtype} B={B} {act}")
        dy = _place(_ints(rng, B, M, dtype, 4), 5, 1) if B != 64 else _ints(rng, B, M, dtype, 4)
        a = torch.from_numpy(2.0 ** rng.integers(-1, 2, M)).float().cuda()
        zp = api.act_pack(_ints(rng, B, M, dtype))
        xp = api.act_pack(_ints(rng, B, N, dtype))
        z, x = api.act_unpack(zp, torch.float32).double(), api.act_unpack(xp, torch.float32).double()
        g, s, gx, gw = _grad_reference(w, dy, a, act, z, x, dtype, False)
        dx, dw, db = w.backward(dy, row_scale=a, act=act, z=zp, x=xp)
        torch.cuda.synchronize()
        assert torch.equal(db.double(), g.sum(0))
        assert torch.equal(dx, gx.to(dtype))
        assert torch.equal(dw, gw.to(dtype))
        # each alone gives the same
        only = w.backward(dy, row_scale=a, act=act, z=zp, dbias=False)
        assert only[1] is None and only[2] is None and torch.equal(only[0], dx)
        only = w.backward(dy, row_scale=a, act=act, z=zp, x=xp, dx=False, dbias=False)
        assert only[0] is None and torch.equal(only[1], dw)
        only = w.backward(dy, row_scale=a, act=act, z=zp, dx=False)
        assert only[0] is None and only[1] is None and torch.equal(only[2], db)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,k,V,T,M,N,B", [
    (16, 2, 1, 256, 2048, 2048, 509), (16, 2, 2, 256, 4096, 1024, 2048),
    (16, 3, 1, 256, 1031, 4096, 1025)])
def test_backward_exact_large(L, k, V, T, M, N, B, dtype):
    _say(f"backward exact large M={M} N={N} B={B} {dtype}")
    rng = np.random.default_rng(B)
    w = Coded(B, M, N, L, k, V, T, dtype, True)
    dy = _ints(rng, B, M, dtype, 2)
    zp, xp = api.act_pack(_ints(rng, B, M, dtype)), api.act_pack(_ints(rng, B, N, dtype))
    z, x = api.act_unpack(zp, torch.float32).double(), api.act_unpack(xp, torch.float32).double()
    g, s, gx, gw = _grad_reference(w, dy, None, "relu", z, x, dtype, False)
    dx, dw, db = w.backward(dy, act="relu", z=zp, x=xp)
    torch.cuda.synchronize()
    assert torch.equal(db.double(), g.sum(0))
    assert torch.equal(dx, gx.to(dtype))
    assert torch.equal(dw, gw.to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape,B", [(SHAPES[0], 37), (SHAPES[1], 128), (SHAPES[6], 9)])
def test_backward_within_bounds(oracle_lib, shape, B, act, dtype):
    import oracle
    L, k, V, T, M, N = shape
    _say(f"backward bounds {shape} B={B} {act} {dtype}")
    rng = np.random.default_rng(N + B)
    w = Coded(N, M, N, L, k, V, T, dtype, False, oracle)

    def normal(*size):
        return torch.from_numpy(rng.standard_normal(size)).to(dtype).cuda()
    dy = normal(B, M)
    a = torch.from_numpy(rng.standard_normal(M) / np.sqrt(N)).float().cuda()
    zp, xp = api.act_pack(normal(B, M)), api.act_pack(normal(B, N))
    z, x = api.act_unpack(zp, torch.float32).double(), api.act_unpack(xp, torch.float32).double()
    # x as the product reads it: rounded to the type (exact but for fp16 values of codes
    # packed from other types, which do not occur here)
    g, s, gx, gw = _grad_reference(w, dy, a, act, z, x, dtype, False)
    dx, dw, db = w.backward(dy, row_scale=a, act=act, z=zp, x=xp)
    torch.cuda.synchronize()
    eg = dy.double().abs() * lc.slope_error(z, act) + 2 * lc.U * g.abs()
    es = eg * a.double().abs() + 2 * lc.U * s.abs()
    es = es + lc.half(dtype) * (s.abs() + es) + lc.tiny(dtype)
    bdb = eg.sum(0) + lc.gamma(B) * (g.abs() + eg).sum(0)
    bdx = es @ w.W.abs() + lc.gamma(M, dtype) * ((s.abs() + es) @ w.W.abs())
    bdx = bdx + lc.half(dtype) * (gx.abs() + bdx) + lc.tiny(dtype)
    bdw = es.t() @ x.abs() + lc.gamma(B, dtype) * ((s.abs() + es).t() @ x.abs())
    bdw = bdw + lc.half(dtype) * (gw.abs() + bdw) + lc.tiny(dtype)
    r = [float(((got.double() - want).abs() / lim).max())
         for got, want, lim in ((db, g.sum(0), bdb), (dx, gx, bdx), (dw, gw, bdw))]
    _say(f"  worst error / bound: dbias {r[0]:.3g}, dx {r[1]:.3g}, dw {r[2]:.3g}")
    assert max(r) <= 1


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,k,V,T,M,N,B", [
    (16, 2, 1, 256, 2047, 2048, 1001), (16, 2, 1, 256, 1023, 2048, 1500),
    (16, 1, 1, 17, 2047, 17 * 121, 1001)])
def test_exact_middle_sizes(L, k, V, T, M, N, B, dtype):
    """Sizes between few tiles and many, where each of the three products is split over its
    sum in some type: forward and backward."""
    _say(f"exact middle sizes M={M} N={N} B={B} {dtype}")
    rng = np.random.default_rng(M + B)
    w = Coded(B, M, N, L, k, V, T, dtype, True)
    x = _ints(rng, B, N, dtype)
    _exact_forward(w, x, rng, dtype, "relu", True, True)
    dy = _ints(rng, B, M, dtype, 2)
    zp, xp = api.act_pack(_ints(rng, B, M, dtype)), api.act_pack(x)
    z, xv = api.act_unpack(zp, torch.float32).double(), api.act_unpack(xp, torch.float32).double()
    g, s, gx, gw = _grad_reference(w, dy, None, "relu", z, xv, dtype, False)
    dx, dw, db = w.backward(dy, act="relu", z=zp, x=xp)
    torch.cuda.synchronize()
    assert torch.equal(db.double(), g.sum(0))
    assert torch.equal(dx, gx.to(dtype))
    assert torch.equal(dw, gw.to(dtype))


def test_threads_with_tables_of_two_sizes():
    """Two host threads on their own streams call one kernel at once, one with a table that
    takes 128 KiB of LDS and one with a table of 2 KiB: both are launched, and right."""
    import threading
    dtype = torch.bfloat16
    M, N = 64, 512
    ws = [Coded(L, M, N, L, 2, 1, 256, dtype, True) for L in (16, 10)]
    cases = [[(w, x, (x.double() @ w.W.t()).to(dtype)) for x in
              (_ints(np.random.default_rng(B), B, N, dtype) for B in (3, 150))] for w in ws]
    torch.cuda.synchronize()
    errs = []

    def work(mine):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(200):
                    for w, x, want in mine:
                        y = w.linear(x)
                for w, x, want in mine:
                    assert torch.equal(w.linear(x), want)
                s.synchronize()
        except Exception as e:  # reported below
            errs.append(e)
    ths = [threading.Thread(target=work, args=(mine,)) for mine in cases]
    for t in ths:
        t.start()
    for t in ths:
        t.join(timeout=60)
    assert not any(t.is_alive() for t in ths) and not errs, errs


@pytest.mark.parametrize("dtype", TYPES)
def test_backward_relu_selects(dtype):
    """Infinite and NaN dy at closed units leave no trace; a checkpoint group of z that
    holds an infinity gives NaN, and no other group does."""
    M, N, B = 96, 256, 40
    w = Coded(8, M, N, 16, 2, 1, 256, dtype, True)
    rng = np.random.default_rng(9)
    z = torch.from_numpy(rng.choice([-2.0, -1.0, 0.0, 1.0, 2.0], size=(B, M))).to(dtype).cuda()
    dy = _ints(rng, B, M, dtype)
    x = _ints(rng, B, N, dtype)
    clean = torch.where(z > 0, dy, torch.zeros_like(dy))
    bad = torch.tensor([float("inf"), float("-inf"), float("nan")], dtype=dtype, device="cuda")
    dy = torch.where(z > 0, dy, bad[torch.arange(M, device="cuda") % 3].expand(B, M))
    xp = api.act_pack(x)
    xv = api.act_unpack(xp, torch.float32).double()
    dx, dw, db = w.backward(dy, act="relu", z=api.act_pack(z), x=xp)
    s = clean.double()
    # integers and multiples of 1/8: every sum is an fp32 number in any order
    assert torch.equal(dx, (s @ w.W).to(dtype))
    assert torch.equal(dw, (s.t() @ xv).to(dtype))
    assert torch.equal(db, s.sum(0).float())
    z[3, 40] = float("inf")                       # columns 32 .. 63 of row 3
    dx, dw, db = w.backward(dy, act="relu", z=api.act_pack(z), x=xp)
    lost = (torch.arange(M, device="cuda") // 32) == 1
    assert torch.equal(torch.isnan(db), lost)
    assert torch.equal(torch.isnan(dx).all(1), torch.arange(B, device="cuda") == 3)
    assert torch.equal(torch.isnan(dw).all(1), lost) and not torch.isnan(dw[~lost]).any()
    rows = torch.arange(B, device="cuda") != 3
    assert torch.equal(dx[rows], (s @ w.W).to(dtype)[rows])


def test_gradients_against_differences():
    """fp32: the gradients of sum(y G) in x, W_hat and bias against central differences of
    the float64 layer.  x is a small integer, which its checkpoint holds exactly; z is not
    (|z| > 127/32 in units of 1/32), so the layer that is differentiated has a constant
    added to z that moves it onto the checkpoint's value, where the slope is taken."""
    L, k, V, T, M, N, B = 8, 2, 1, 16, 6, 16, 3
    rng = np.random.default_rng(8)
    dt = torch.float32
    w = Coded(1, M, N, L, k, V, T, dt, True)
    x = _ints(rng, B, N, dt, 1)
    bias = torch.from_numpy(rng.integers(-8, 9, M) / 8.0).float().cuda()
    a = torch.full((M,), 0.25, device="cuda")
    G = torch.from_numpy(rng.standard_normal((B, M))).to(dt).cuda()
    for act in ("silu", "gelu"):
        z = (x.double() @ w.W.t()) * 0.25 + bias.double()
        _, pre = w.linear(x, row_scale=a, bias=bias, act=act, pre=True)
        assert torch.equal(pre.double(), z)
        zp, xp = api.act_pack(pre), api.act_pack(x)
        assert torch.equal(api.act_unpack(xp, dt), x)
        shift = api.act_unpack(zp, dt).double() - z
        assert float(shift.abs().max()) <= 1 / 32  # half a step of 1/16
        dx, dw, db = w.backward(G, row_scale=a, act=act, z=zp, x=xp)

        def loss(xx, ww, bb):
            return float((lc.act((xx @ ww.t()) * 0.25 + bb + shift, act) * G.double()).sum())
        h = 1e-4
        args = [x.double(), w.W.clone(), bias.double()]
        for n, grad in ((0, dx), (1, dw), (2, db)):
            for _ in range(6):
                at = tuple(rng.integers(0, d) for d in args[n].shape)
                lo, hi = [t.clone() for t in args], [t.clone() for t in args]
                lo[n][at] -= h
                hi[n][at] += h
                diff = (loss(*hi) - loss(*lo)) / (2 * h)
                # third derivative of the loss along one argument: |act'''| <= 2, |x| and
                # |W| at most 4, sums of B M terms of |G| below 4
                trunc = h * h / 6 * 2 * 4 ** 3 * B * M * 4
                assert abs(float(grad[at]) - diff) <= trunc + 1e-5 * max(1, abs(diff)) * 4


@pytest.mark.parametrize("dtype", TYPES)
def test_encode_then_train_step(dtype):
    """The pieces as they are used together: a weight matrix is encoded with the layer's
    table, the layer runs forward keeping z, z and x are packed, the backward pass reads
    them; against the same step in float64 from the decoded matrix."""
    L, k, V, T, M, N, B = 16, 2, 1, 256, 24, 512, 48
    _say(f"encode and train step {dtype}")
    W, _ = wl.random_small(3, M, N, False)
    table = api.make_codebook(L, V, 3001).to(dtype)
    Wn = torch.from_numpy(W).cuda()
    a, _, _ = api.scale_field(Wn, normalized=False)
    enc = api.encode(Wn / a[:, None], None, table.float(), L, k, V, T, recon=True)
    w = Coded.__new__(Coded)
    w.shape, w.bits, w.s0, w.table = (M, N, L, k, V, T), enc.bitstream, enc.start_state, table
    w.W = enc.recon.double()
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.standard_normal((B, N))).to(dtype).cuda()
    bias = torch.from_numpy(rng.standard_normal(M)).float().cuda()
    y, pre = w.linear(x, row_scale=a, bias=bias, act="gelu", pre=True)
    zp, xp = api.act_pack(pre), api.act_pack(x)
    del pre
    dy = (y.float() * 0.5).to(dtype)
    dx, dw, db = w.backward(dy, row_scale=a, act="gelu", z=zp, x=xp)
    torch.cuda.synchronize()
    ez, ey, mag = lc.forward(w.W, x.double(), a.double(), bias.double(), "gelu", None)
    _, lim = lc.forward_bounds(ez, ey, mag, None, "gelu", N, dtype)
    assert bool(((y.double() - ey).abs() <= lim).all())
    z = api.act_unpack(zp, torch.float32).double()
    # the checkpoint of z is within one step of z, itself rounded to the type
    step = torch.ldexp(torch.ones_like(zp.scale, dtype=torch.float64), zp.scale.int() - 133)
    step = step.repeat_interleave(32, 1)[:, :M]
    dz, _ = lc.forward_bounds(ez, ey, mag, None, "gelu", N, dtype)
    assert bool(((z - ez).abs() <= step + dz).all())
    xv = api.act_unpack(xp, torch.float32).double()
    g, s, gx, gw = _grad_reference(w, dy, a, "gelu", z, xv, dtype, False)
    u = 4 * lc.half(dtype) + 64 * lc.U
    assert bool(((db.double() - g.sum(0)).abs() <= 64 * lc.U * g.abs().sum(0) + 1e-12).all())
    assert bool(((dx.double() - gx).abs() <= u * (s.abs() @ w.W.abs()) + 1e-6).all())
    assert bool(((dw.double() - gw).abs() <= u * (s.abs().t() @ xv.abs()) + 1e-6).all())


@pytest.mark.parametrize("B", [1, 20, 700])
def test_stream_and_repeats(B):
    """On another stream, and twice: the same bits."""
    dtype = torch.bfloat16
    w = Coded(2, 512, 1024, 16, 2, 1, 256, dtype, False)
    rng = np.random.default_rng(B)
    x = torch.from_numpy(rng.standard_normal((B, 1024))).to(dtype).cuda()
    dy = torch.from_numpy(rng.standard_normal((B, 512))).to(dtype).cuda()
    xp, zp = api.act_pack(x), api.act_pack(dy)

    def once():
        return [w.linear(x, act="silu"), *w.backward(dy, act="silu", z=zp, x=xp)]
    first = once()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        second = once()
    s.synchronize()
    third = once()
    torch.cuda.synchronize()
    for p, q, r in zip(first, second, third):
        assert torch.equal(p, q) and torch.equal(p, r)


@pytest.mark.parametrize("B", [1, 24, 520])
def test_captured_and_replayed(B):
    """Two captured graphs, each with its own workspace, replayed in turn with eager calls
    between: every replay equals the eager result on the inputs of the moment."""
    dtype = torch.bfloat16
    M, N = 384, 1024
    w = Coded(4, M, N, 16, 2, 1, 256, dtype, False)
    g = torch.Generator("cuda").manual_seed(B)
    x = torch.randn(B, N, generator=g, device="cuda").to(dtype)
    dy = torch.randn(B, M, generator=g, device="cuda").to(dtype)

    def both():
        y, z = w.linear(x, act="gelu", pre=True)
        zp, xp = api.act_pack(z), api.act_pack(x)
        return [y, *w.backward(dy, act="gelu", z=zp, x=xp)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = both()
        graphs.append((graph, outs))
    for turn in range(3):
        x.copy_(torch.randn(B, N, generator=g, device="cuda"))
        want = both()
        torch.cuda.synchronize()
        for graph, outs in graphs:
            for o in outs:
                o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for p, q in zip(outs, want):
                assert torch.equal(p, q), f"turn {turn}"
            both()
            torch.cuda.synchronize()


def test_given_workspace_and_refusals():
    dtype = torch.float16
    M, N, B = 64, 512, 300
    w = Coded(5, M, N, 16, 2, 1, 256, dtype, True)
    x = _ints(np.random.default_rng(0), B, N, dtype)
    need = _lib.tcq_decode_linear_workspace_bytes(_lib.TCQ_F16, B, *w.shape)
    y = w.linear(x, workspace=api.Workspace(need))
    assert torch.equal(y, (x.double() @ w.W.t()).to(dtype))
    if need:
        with pytest.raises(_lib.TcqError) as e:
            w.linear(x, workspace=api.Workspace(need - 1))
        assert e.value.status == _lib.TCQ_EWORKSPACE
    with pytest.raises(AssertionError):
        w.linear(x.float())                       # codebook of another type
    with pytest.raises(AssertionError):
        w.linear(x.t())                           # columns contiguous
    with pytest.raises(AssertionError):
        w.linear(x, bias=torch.zeros(M, device="cuda", dtype=dtype))
    with pytest.raises(KeyError):
        w.linear(x, act="tanh")
    with pytest.raises(AssertionError):
        w.backward(x[:, :M].contiguous(), act="gelu")   # no checkpoint of z
    with pytest.raises(AssertionError):
        w.backward(x[:, :M].contiguous(), dx=False, dbias=False)
