"""Argument checks of the coded linear layer and the checkpoints: bad calls are rejected
before anything reaches a GPU (no device work is issued by these tests)."""
import ctypes

import numpy as np
import pytest

import trellis_coded_bit_amd as tcq
from trellis_coded_bit_amd import _lib

import linear_check as lc

FAKE = 0x7F0000001000  # never dereferenced: every call below fails validation first
E = _lib
BIG = 1 << 45


def _linear(**kw):
    a = dict(bits=FAKE, s0=FAKE, cb=FAKE, M=4, N=512, L=16, k=2, V=1, T=256, dtype=E.TCQ_BF16,
             x=FAKE, B=3, ldx=512, a=None, b=None, act=0, res=None, ldr=4, y=FAKE, ldy=4,
             pre=None, ldp=4, ws=None, wsb=BIG)
    a.update(kw)
    return _lib.load().tcq_decode_linear(*a.values(), None)


def test_decode_linear_argument_checks():
    assert _linear(N=500) == E.TCQ_EINVAL
    assert _linear(B=-1) == E.TCQ_EINVAL
    assert _linear(M=-1) == E.TCQ_EINVAL
    assert _linear(L=20) == E.TCQ_EUNSUPPORTED
    assert _linear(dtype=3) == E.TCQ_EINVAL
    assert "dtype" in tcq.tcq_last_error()
    assert _linear(act=4) == E.TCQ_EINVAL
    assert _linear(act=-1) == E.TCQ_EINVAL
    assert _linear(x=None) == E.TCQ_EINVAL
    assert _linear(y=None) == E.TCQ_EINVAL
    assert _linear(cb=None) == E.TCQ_EINVAL
    assert _linear(bits=None) == E.TCQ_EINVAL
    assert _linear(ldx=511) == E.TCQ_EINVAL
    assert _linear(ldy=3) == E.TCQ_EINVAL
    assert _linear(res=FAKE, ldr=3) == E.TCQ_EINVAL
    assert _linear(res=FAKE, ldr=5) == E.TCQ_EINVAL          # in place of y, other stride
    assert _linear(pre=FAKE + 4096, ldp=3) == E.TCQ_EINVAL
    assert _linear(pre=FAKE) == E.TCQ_EINVAL                 # pre in place of y
    assert _linear(x=FAKE + 1) == E.TCQ_EINVAL               # not aligned to its values
    assert "aligned" in tcq.tcq_last_error()
    assert _linear(dtype=E.TCQ_F32, cb=FAKE + 2) == E.TCQ_EINVAL
    assert _linear(M=(1 << 21) + 1, ldy=1 << 22) == E.TCQ_EUNSUPPORTED
    assert _linear(B=(1 << 23) + 1) == E.TCQ_EUNSUPPORTED
    assert "limits" in tcq.tcq_last_error()
    # a large batch needs a workspace
    big = dict(B=4096, M=4096, ldy=4096)
    assert _linear(**big) == E.TCQ_EWORKSPACE
    assert _linear(**big, ws=FAKE, wsb=16) == E.TCQ_EWORKSPACE
    assert _linear(**big, ws=FAKE + 8) == E.TCQ_EINVAL
    assert "256-byte" in tcq.tcq_last_error()
    # nothing to do
    assert _linear(B=0) == E.TCQ_OK
    assert _linear(M=0) == E.TCQ_OK
    assert tcq.tcq_last_error() == ""


def _backward(**kw):
    a = dict(bits=FAKE, s0=FAKE, cb=FAKE, M=4, N=512, L=16, k=2, V=1, T=256, dtype=E.TCQ_F16,
             dy=FAKE, B=3, lddy=4, a=None, act=E.TCQ_ACT_GELU, zq=FAKE, ldz=4, ze=FAKE,
             xq=FAKE, ldxq=512, xe=FAKE, dx=FAKE, lddx=512, dw=FAKE, lddw=512, db=FAKE, ws=FAKE,
             wsb=16)
    a.update(kw)
    return _lib.load().tcq_decode_linear_backward(*a.values(), None)


def test_decode_linear_backward_argument_checks():
    assert _backward() == E.TCQ_EWORKSPACE
    assert _backward(N=500) == E.TCQ_EINVAL
    assert _backward(dtype=-1) == E.TCQ_EINVAL
    assert _backward(act=9) == E.TCQ_EINVAL
    assert _backward(B=-2) == E.TCQ_EINVAL
    assert _backward(dx=None, dw=None, db=None) == E.TCQ_EINVAL
    assert "none of" in tcq.tcq_last_error()
    assert _backward(dy=None) == E.TCQ_EINVAL
    assert _backward(lddy=3) == E.TCQ_EINVAL
    assert _backward(zq=None) == E.TCQ_EINVAL
    assert _backward(ze=None) == E.TCQ_EINVAL
    assert _backward(ldz=2) == E.TCQ_EINVAL
    assert _backward(xq=None) == E.TCQ_EINVAL
    assert _backward(xe=None) == E.TCQ_EINVAL
    assert _backward(ldxq=100) == E.TCQ_EINVAL
    assert _backward(lddx=100) == E.TCQ_EINVAL
    assert _backward(lddw=100) == E.TCQ_EINVAL
    assert _backward(cb=None) == E.TCQ_EINVAL
    assert _backward(dw=FAKE + 1) == E.TCQ_EINVAL
    assert _backward(L=17) == E.TCQ_EUNSUPPORTED
    # what is not wanted is not asked for
    assert _backward(zq=None, ze=None, act=E.TCQ_ACT_NONE) == E.TCQ_EWORKSPACE
    assert _backward(xq=None, xe=None, dw=None) == E.TCQ_EWORKSPACE
    assert _backward(bits=None, s0=None, cb=None, dx=None) == E.TCQ_EWORKSPACE
    assert _backward(ws=FAKE + 16, wsb=BIG) == E.TCQ_EINVAL


def test_workspace_queries():
    lib = _lib.load()
    b = ctypes.c_size_t(123)
    ref = ctypes.byref(b)
    assert lib.tcq_decode_linear_workspace_bytes(1, 0, 64, 512, 16, 2, 1, 256, ref) == E.TCQ_OK
    assert b.value == 0
    assert lib.tcq_decode_linear_workspace_bytes(1, 4, 64, 512, 16, 2, 1, 256, None) == \
        E.TCQ_EINVAL
    assert lib.tcq_decode_linear_workspace_bytes(7, 4, 64, 512, 16, 2, 1, 256, ref) == \
        E.TCQ_EINVAL
    need = _lib.tcq_decode_linear_workspace_bytes(E.TCQ_BF16, 8192, 4096, 14336, 16, 3, 1, 256)
    assert need < 1 << 40
    every = _lib.tcq_decode_linear_backward_workspace_bytes(E.TCQ_F32, 100, 64, 512, 16, 2, 1,
                                                            256, True, True, True)
    some = _lib.tcq_decode_linear_backward_workspace_bytes(E.TCQ_F32, 100, 64, 512, 16, 2, 1,
                                                           256, False, True, False)
    assert some < every
    assert lib.tcq_decode_linear_backward_workspace_bytes(0, 4, 64, 512, 16, 2, 1, 256, 1, 1, 1,
                                                          None) == E.TCQ_EINVAL


def test_checkpoint_argument_checks():
    lib = _lib.load()

    def pack(**kw):
        a = dict(X=FAKE, dtype=E.TCQ_BF16, rows=4, cols=64, ldx=64, codes=FAKE, ldq=64,
                 scale=FAKE)
        a.update(kw)
        return lib.tcq_act_pack(*a.values(), None)

    assert pack(dtype=5) == E.TCQ_EINVAL
    assert pack(rows=-1) == E.TCQ_EINVAL
    assert pack(cols=1 << 31) == E.TCQ_EUNSUPPORTED
    assert pack(X=None) == E.TCQ_EINVAL
    assert pack(X=FAKE + 1) == E.TCQ_EINVAL
    assert pack(codes=None) == E.TCQ_EINVAL
    assert pack(scale=None) == E.TCQ_EINVAL
    assert pack(ldx=63) == E.TCQ_EINVAL
    assert pack(ldq=63) == E.TCQ_EINVAL
    assert pack(rows=0) == E.TCQ_OK
    assert pack(cols=0) == E.TCQ_OK

    def unpack(**kw):
        a = dict(codes=FAKE, ldq=64, scale=FAKE, rows=4, cols=64, dtype=E.TCQ_F32, out=FAKE,
                 ldo=64)
        a.update(kw)
        return lib.tcq_act_unpack(*a.values(), None)

    assert unpack(dtype=5) == E.TCQ_EINVAL
    assert unpack(codes=None) == E.TCQ_EINVAL
    assert unpack(out=None) == E.TCQ_EINVAL
    assert unpack(out=FAKE + 2) == E.TCQ_EINVAL
    assert unpack(ldo=63) == E.TCQ_EINVAL
    assert unpack(rows=0) == E.TCQ_OK
    with pytest.raises(tcq.TcqError) as e:
        tcq.tcq_act_unpack(FAKE, 3, FAKE, 4, 64, E.TCQ_F32, FAKE, 64, None)
    assert e.value.status == E.TCQ_EINVAL and "tcq_act_unpack" in str(e.value)


def test_reference_slopes_are_the_activations_derivatives():
    """The formulas the GPU tests use, against central differences in float64."""
    torch = pytest.importorskip("torch")
    z = torch.linspace(-6, 6, 241, dtype=torch.float64) + 0.013
    h = 1e-5
    for name in ("none", "relu", "silu", "gelu"):
        diff = (lc.act(z + h, name) - lc.act(z - h, name)) / (2 * h)
        # third derivatives are below 2: h^2 / 3 truncation, and rounding of act over 2 h
        assert float((lc.slope(z, name) - diff).abs().max()) < h * h + 4 * 2.0 ** -53 * 7 / h


def test_reference_checkpoint_round_trip():
    """The reference pack: values that are multiples of their group's step come back."""
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(0)
    q = rng.integers(-127, 128, size=(5, 70)).astype(float)
    q[:, ::32] = 127  # pins every group's exponent
    codes, scale = lc.pack(torch.from_numpy(q * 0.25))
    assert np.array_equal(codes, q) and np.array_equal(lc.unpack(codes, scale), q * 0.25)
    # a planted mistake: one exponent off is seen
    assert not np.array_equal(lc.unpack(codes, scale + 1), q * 0.25)
