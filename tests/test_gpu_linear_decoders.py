"""The coded linear layer over every (k V, V) that its decoders are compiled for: each has word
counts, shifts and table parts of its own.  Exact inputs (see test_gpu_linear.py), against the
oracle's decode."""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import api  # noqa: E402

from test_gpu_linear import Coded, _exact_forward, _ints  # noqa: E402

TYPES = [torch.float32, torch.float16, torch.bfloat16]


def _say(msg):
    sys.stdout.write(msg + "\n")
    sys.stdout.flush()


# L, k, V, T, M, N: tables of one part and several; blocks of 8, 12 (no power of two) and 20
# chunks; V = 3 and kV = 5 and 7, which take the generic decoder
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [
    (16, 1, 4, 64, 40, 192), (12, 1, 4, 96, 33, 288), (16, 1, 4, 160, 17, 320),
    (16, 6, 1, 64, 40, 128), (11, 6, 1, 24, 37, 120), (16, 3, 2, 64, 40, 192),
    (10, 3, 2, 96, 21, 192), (16, 8, 1, 64, 33, 128), (9, 8, 1, 40, 50, 120),
    (16, 4, 2, 64, 40, 128), (13, 4, 2, 96, 19, 96), (16, 2, 4, 96, 35, 192),
    (16, 4, 1, 96, 40, 288), (16, 2, 2, 96, 34, 192), (16, 1, 2, 32, 40, 224),
    (16, 5, 1, 64, 33, 128), (14, 7, 1, 64, 18, 64), (16, 2, 3, 48, 20, 96)])
def test_every_decoder(oracle_lib, shape, dtype):
    import oracle
    L, k, V, T, M, N = shape
    rng = np.random.default_rng(L * 1000 + k * 100 + V * 10 + T)
    w = Coded(M * N, M, N, L, k, V, T, dtype, True, oracle)
    for B in (1, 16, 17, 60, 65, 128, 129, 200):
        _say(f"decoders {shape} {dtype} B={B}")
        _exact_forward(w, _ints(rng, B, N, dtype), rng, dtype, "relu", B % 2 == 0, False)
    # the matrix alone: dx of the identity
    eye = torch.eye(M, dtype=dtype, device="cuda")
    dx = w.backward(eye, dbias=False)[0]
    assert torch.equal(dx.double(), w.W)
    # all bits set and all clear, at either end of the start states
    for fill, s0 in ((-1, (1 << (L - k * V)) - 1), (0, 0)):
        w.bits.fill_(fill)
        tail = k * T % 32
        if tail and fill:
            w.bits[:, -1] = -(1 << (32 - tail))
        w.s0.fill_(s0)
        want = api.decode(w.bits, w.s0, w.table.float(), M, N, L, k, V, T)
        assert torch.equal(w.backward(eye, dbias=False)[0].float(), want)
        x = _ints(rng, 20, N, dtype)
        assert torch.equal(w.linear(x), (x.double() @ want.double().t()).to(dtype))
