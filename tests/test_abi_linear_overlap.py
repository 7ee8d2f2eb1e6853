"""Outputs of the coded linear layer and the checkpoints over their inputs or one another are
refused before anything reaches a GPU (every call here fails), and columns of one buffer
side by side are not (checked on the comparison itself, tests/region_check.cpp)."""
import os
import subprocess

import trellis_coded_bit_amd as tcq
from trellis_coded_bit_amd import _lib

E = _lib
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
AT = 0x7F0000000000  # addresses below are never dereferenced: every call fails validation
FAR = AT + (1 << 30)
WS = AT + (1 << 40)


def test_regions(tmp_path):
    exe = tmp_path / "regions"
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-I",
                    os.path.join(ROOT, "trellis_coded_bit_amd", "csrc"),
                    os.path.join(ROOT, "tests", "region_check.cpp"), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "regions ok" in res.stdout


def _refused(names, **kw):
    a = dict(bits=AT, s0=AT, cb=AT, M=512, N=512, L=16, k=2, V=1, T=256, dtype=E.TCQ_BF16,
             x=AT, B=300, ldx=512, a=None, b=None, act=0, res=None, ldr=512, y=FAR, ldy=512,
             pre=None, ldp=512, ws=WS, wsb=1 << 40)
    a.update(kw)
    assert _lib.load().tcq_decode_linear(*a.values(), None) == E.TCQ_EINVAL, kw
    assert names in tcq.tcq_last_error()


def test_linear_outputs_over_inputs():
    last = 2 * (299 * 512 + 511)
    for y in (AT, AT + 2, AT + last):
        _refused("y and x overlap", y=y)
    _refused("y and x overlap", x=AT + last, y=AT)
    _refused("y and x overlap", y=AT, B=1)                    # without a workspace too
    _refused("y and x overlap", y=AT, res=AT)
    _refused("pre and x overlap", pre=AT)
    _refused("pre and y overlap", pre=FAR + 2)
    _refused("y and residual overlap", res=FAR + 2)
    _refused("pre and residual overlap", res=AT + (1 << 29), pre=AT + (1 << 29) + 1024 * 7)


def test_linear_columns_of_one_buffer():
    ld = dict(ldx=2048, ldy=2048, ldr=2048, ldp=2048)
    _refused("y and x overlap", y=AT + 2 * 511, **ld)
    _refused("y and x overlap", y=AT + 2 * (2048 * 40 + 511), **ld)
    _refused("y and x overlap", y=AT + 2 * (2048 * 40 - 511), **ld)
    _refused("y and x overlap", x=AT + 2 * (2048 * 40 - 511), y=AT, **ld)
    # row i of y starts at column 700 - i of x's buffer: 511 at i = 189
    _refused("y and x overlap", y=AT + 2 * 700, ldx=2048, ldy=2047)


def test_gradients_over_one_another():
    def refused(names, **kw):
        a = dict(bits=AT, s0=AT, cb=AT, M=64, N=512, L=16, k=2, V=1, T=256, dtype=E.TCQ_F16,
                 dy=AT, B=30, lddy=64, a=None, act=0, zq=None, ldz=64, ze=None, xq=AT,
                 ldxq=512, xe=AT, dx=AT + (1 << 20), lddx=512, dw=AT + (2 << 20), lddw=512,
                 db=AT + (3 << 20), ws=WS, wsb=1 << 40)
        a.update(kw)
        assert _lib.load().tcq_decode_linear_backward(*a.values(), None) == E.TCQ_EINVAL
        assert names in tcq.tcq_last_error()
    refused("dx and dw overlap", dw=AT + (1 << 20))
    refused("dx and dbias overlap", db=AT + (1 << 20) + 2 * 30 * 512 - 4)
    refused("dw and dbias overlap", db=AT + (2 << 20) - 4 * 63)


def test_checkpoints_over_their_inputs():
    lib = _lib.load()

    def pack(X=AT, codes=FAR, scale=WS):
        return lib.tcq_act_pack(X, E.TCQ_BF16, 4, 64, 64, codes, 64, scale, None)

    def unpack(codes=AT, scale=FAR, out=WS):
        return lib.tcq_act_unpack(codes, 64, scale, 4, 64, E.TCQ_F32, out, 64, None)
    for rc in (pack(codes=AT), pack(codes=AT + 511), pack(scale=AT + 100), pack(scale=FAR + 255),
               unpack(out=AT), unpack(out=AT - 4 * 255), unpack(out=FAR - 8)):
        assert rc == E.TCQ_EINVAL and "overlap" in tcq.tcq_last_error()
