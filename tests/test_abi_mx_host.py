"""Argument checks of the microscaled operators: bad calls are rejected before anything reaches a
GPU (no device work is issued by these tests)."""
import ctypes

import pytest

import trellis_coded_bit_amd as tcq
from trellis_coded_bit_amd import _lib

E = _lib
FAKE = 0x7F0000001000  # never dereferenced: every call below fails validation or has no work
FAR = 1 << 32          # apart from FAKE
BIG = 1 << 45


def _pack(**kw):
    a = dict(X=FAKE, dtype=E.TCQ_BF16, rows=4, cols=70, ldx=70, fmt=E.TCQ_FP4, codes=FAKE + FAR,
             ldq=48, scale=FAKE + 2 * FAR)
    a.update(kw)
    return _lib.load().tcq_mx_pack(*a.values(), None)


def _unpack(**kw):
    a = dict(codes=FAKE, ldq=96, scale=FAKE + FAR, rows=4, cols=70, fmt=E.TCQ_FP8,
             dtype=E.TCQ_F16, out=FAKE + 2 * FAR, ldo=70)
    a.update(kw)
    return _lib.load().tcq_mx_unpack(*a.values(), None)


def test_pack_argument_checks():
    assert _pack(fmt=2) == E.TCQ_EINVAL
    assert "TCQ_FP4" in tcq.tcq_last_error()
    assert _pack(dtype=3) == E.TCQ_EINVAL
    assert _pack(rows=-1) == E.TCQ_EINVAL
    assert _pack(cols=-1) == E.TCQ_EINVAL
    assert _pack(rows=1 << 31) == E.TCQ_EUNSUPPORTED
    assert _pack(X=None) == E.TCQ_EINVAL
    assert _pack(X=FAKE + 1) == E.TCQ_EINVAL
    assert _pack(ldx=69) == E.TCQ_EINVAL
    assert _pack(codes=None) == E.TCQ_EINVAL
    assert _pack(scale=None) == E.TCQ_EINVAL
    assert _pack(ldq=47) == E.TCQ_EINVAL
    assert _pack(ldq=32) == E.TCQ_EINVAL              # three groups are 48 bytes
    assert "whole groups" in tcq.tcq_last_error()
    assert _pack(codes=FAKE + FAR + 8) == E.TCQ_EINVAL
    assert "16 bytes" in tcq.tcq_last_error()
    assert _pack(codes=FAKE) == E.TCQ_EINVAL          # over X
    assert "overlap" in tcq.tcq_last_error()
    assert _pack(scale=FAKE + 4 * 140 - 1) == E.TCQ_EINVAL
    assert _pack(scale=FAKE + FAR + 3 * 48 + 47) == E.TCQ_EINVAL
    assert _pack(rows=0) == E.TCQ_OK and _pack(cols=0) == E.TCQ_OK
    assert tcq.tcq_last_error() == ""


def test_unpack_argument_checks():
    assert _unpack(fmt=-1) == E.TCQ_EINVAL
    assert _unpack(dtype=-1) == E.TCQ_EINVAL
    assert _unpack(cols=1 << 31) == E.TCQ_EUNSUPPORTED
    assert _unpack(ldq=80) == E.TCQ_EINVAL
    assert _unpack(codes=FAKE + 4) == E.TCQ_EINVAL
    assert _unpack(out=None) == E.TCQ_EINVAL
    assert _unpack(ldo=69) == E.TCQ_EINVAL
    assert _unpack(out=FAKE) == E.TCQ_EINVAL
    assert _unpack(out=FAKE + FAR) == E.TCQ_EINVAL
    assert _unpack(rows=0) == E.TCQ_OK


def _linear(**kw):
    a = dict(w=FAKE, ldw=32, ws=FAKE + FAR, M=8, N=64, dtype=E.TCQ_BF16, x=FAKE + 2 * FAR, B=3,
             ldx=64, fmt=E.TCQ_FP8, xq=FAKE + 3 * FAR, ldxq=64, xs=FAKE + 4 * FAR, bias=None,
             res=None, ldr=8, y=FAKE + 5 * FAR, ldy=8, wsp=FAKE + 6 * FAR, wsb=16)
    a.update(kw)
    return _lib.load().tcq_mx_linear(*a.values(), None)


def test_linear_argument_checks():
    assert _linear() == E.TCQ_EWORKSPACE
    assert _linear(wsp=None, wsb=BIG) == E.TCQ_EWORKSPACE
    assert _linear(wsp=FAKE + 8, wsb=BIG) == E.TCQ_EINVAL
    assert _linear(fmt=7) == E.TCQ_EINVAL
    assert _linear(dtype=7) == E.TCQ_EINVAL
    assert _linear(B=-1) == E.TCQ_EINVAL
    assert _linear(M=(1 << 21) + 1, ldy=1 << 22) == E.TCQ_EUNSUPPORTED
    assert _linear(B=(1 << 23) + 1) == E.TCQ_EUNSUPPORTED
    assert _linear(w=None) == E.TCQ_EINVAL
    assert _linear(ws=None) == E.TCQ_EINVAL
    assert _linear(ldw=16) == E.TCQ_EINVAL
    assert _linear(w=FAKE + 2) == E.TCQ_EINVAL
    assert _linear(ldx=63) == E.TCQ_EINVAL
    assert _linear(x=FAKE + 2 * FAR + 1) == E.TCQ_EINVAL
    assert _linear(xs=None) == E.TCQ_EINVAL           # codes kept without their scales
    assert _linear(x=None, xq=None) == E.TCQ_EINVAL   # neither x nor its codes
    assert _linear(ldxq=48) == E.TCQ_EINVAL
    assert _linear(y=None) == E.TCQ_EINVAL
    assert _linear(ldy=7) == E.TCQ_EINVAL
    assert _linear(res=FAKE + 5 * FAR, ldr=9) == E.TCQ_EINVAL
    # outputs over inputs and one another
    ws = dict(wsb=BIG)
    for name in ("x", "w", "ws", "xq", "xs"):
        assert _linear(**{name: FAKE + 5 * FAR}, **ws) == E.TCQ_EINVAL
        assert "overlap" in tcq.tcq_last_error()
    assert _linear(xq=FAKE, **ws) == E.TCQ_EINVAL
    assert _linear(xs=FAKE + 2 * FAR, **ws) == E.TCQ_EINVAL
    assert _linear(xs=FAKE + 3 * FAR, **ws) == E.TCQ_EINVAL
    assert _linear(res=FAKE + 5 * FAR + 2, **ws) == E.TCQ_EINVAL
    # what is not there is not asked for
    assert _linear(xq=None, xs=None) == E.TCQ_EWORKSPACE
    assert _linear(x=None) == E.TCQ_EWORKSPACE
    assert _linear(B=0) == E.TCQ_OK and _linear(M=0) == E.TCQ_OK


def _backward(**kw):
    a = dict(w=FAKE, ldw=32, ws=FAKE + FAR, M=8, N=64, dtype=E.TCQ_F16, dy=FAKE + 2 * FAR, B=3,
             lddy=8, fmt=E.TCQ_FP4, xq=FAKE + 3 * FAR, ldxq=32, xs=FAKE + 4 * FAR,
             dx=FAKE + 5 * FAR, lddx=64, dw=FAKE + 6 * FAR, lddw=64, db=FAKE + 7 * FAR,
             wsp=FAKE + 8 * FAR, wsb=16)
    a.update(kw)
    return _lib.load().tcq_mx_linear_backward(*a.values(), None)


def test_backward_argument_checks():
    assert _backward() == E.TCQ_EWORKSPACE
    assert _backward(dx=None, dw=None, db=None) == E.TCQ_EINVAL
    assert _backward(dy=None) == E.TCQ_EINVAL
    assert _backward(lddy=7) == E.TCQ_EINVAL
    assert _backward(w=None) == E.TCQ_EINVAL
    assert _backward(xq=None) == E.TCQ_EINVAL
    assert _backward(xs=None) == E.TCQ_EINVAL
    assert _backward(ldxq=16) == E.TCQ_EINVAL
    assert _backward(lddx=63) == E.TCQ_EINVAL
    assert _backward(lddw=63) == E.TCQ_EINVAL
    assert _backward(fmt=2) == E.TCQ_EINVAL
    assert _backward(dtype=9) == E.TCQ_EINVAL
    assert _backward(B=-1) == E.TCQ_EINVAL
    assert _backward(w=None, dx=None) == E.TCQ_EWORKSPACE
    assert _backward(xq=None, xs=None, dw=None) == E.TCQ_EWORKSPACE
    ws = dict(wsb=BIG)
    for name in ("dy", "w", "ws", "dw", "db"):
        assert _backward(**{name: FAKE + 5 * FAR}, **ws) == E.TCQ_EINVAL
        assert "overlap" in tcq.tcq_last_error()
    for name in ("xq", "xs", "db"):
        assert _backward(**{name: FAKE + 6 * FAR}, **ws) == E.TCQ_EINVAL


def test_workspace_queries():
    lib = _lib.load()
    b = ctypes.c_size_t(5)
    ref = ctypes.byref(b)
    assert lib.tcq_mx_linear_workspace_bytes(0, 0, 8, 64, ref) == E.TCQ_OK and b.value == 0
    assert lib.tcq_mx_linear_workspace_bytes(0, 4, 8, 64, None) == E.TCQ_EINVAL
    assert lib.tcq_mx_linear_workspace_bytes(3, 4, 8, 64, ref) == E.TCQ_EINVAL
    assert lib.tcq_mx_linear_workspace_bytes(0, 4, 8, -1, ref) == E.TCQ_EINVAL
    assert lib.tcq_mx_linear_backward_workspace_bytes(5, 4, 8, 64, 1, 1, 1, ref) == E.TCQ_EINVAL
    assert lib.tcq_mx_linear_backward_workspace_bytes(0, 4, 8, 64, 1, 1, 1, None) == E.TCQ_EINVAL
    for fmt in (0, 1):
        sizes = [_lib.tcq_mx_linear_workspace_bytes(fmt, B, 4096, 4096)
                 for B in range(1, 3000, 7)]
        assert sizes == sorted(sizes)
    for dtype in (0, 1, 2):
        sizes = [_lib.tcq_mx_linear_backward_workspace_bytes(dtype, B, 1000, 2048, True, True,
                                                             True) for B in range(1, 3000, 7)]
        assert sizes == sorted(sizes)


def test_python_calls_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    from trellis_coded_bit_amd import api
    with pytest.raises(AssertionError):
        api.mx_pack(torch.zeros(2, 32))
    p = api.MxPacked(torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.uint8),
                     32, "fp4")
    with pytest.raises(AssertionError):
        api.mx_unpack(p, torch.float32)
    with pytest.raises(AssertionError):
        api.mx_linear(torch.zeros(2, 32), p)
    with pytest.raises(AssertionError):
        api.mx_linear_backward(torch.zeros(2, 2), p)
