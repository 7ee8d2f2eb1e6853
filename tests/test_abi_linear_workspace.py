"""Workspace sizes of the coded linear layer: one that serves a batch serves every smaller one
(the queries touch no GPU)."""
import numpy as np
import pytest

from trellis_coded_bit_amd import _lib

SHAPES = [(4096, 4096, 16, 2, 1, 256), (14336, 4096, 16, 2, 2, 256), (4096, 14336, 16, 3, 1, 256),
          (2048, 2048, 16, 2, 1, 256), (64, 512, 16, 2, 1, 256), (130, 17 * 9, 16, 1, 1, 17),
          (1, 64, 8, 2, 1, 64), (1031, 4160, 12, 2, 1, 64), (300, 500, 8, 1, 1, 20)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [_lib.TCQ_F32, _lib.TCQ_F16, _lib.TCQ_BF16])
def test_need_grows_with_the_batch(shape, dtype):
    M, N, L, k, V, T = shape
    rng = np.random.default_rng(M)
    batches = sorted({*range(0, 300), 511, 512, 513, 1023, 1024, 1025, 2048, 4096, 8192, 16384,
                      *(int(b) for b in np.exp(rng.uniform(5, 11, 200)))})
    need = [_lib.tcq_decode_linear_workspace_bytes(dtype, B, *shape) for B in batches]
    assert need == sorted(need)
    for wanted in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)):
        need = [_lib.tcq_decode_linear_backward_workspace_bytes(dtype, B, *shape, *wanted)
                for B in batches]
        assert need == sorted(need), wanted


def test_need_stays_near_the_buffers():
    """The matrix, x and at most 32 MiB of shares (fp32 sums of products split over k)."""
    for dtype, size in ((_lib.TCQ_F32, 4), (_lib.TCQ_BF16, 2)):
        for B in (300, 2048, 8192):
            for M, N, L, k, V, T in SHAPES:
                need = _lib.tcq_decode_linear_workspace_bytes(dtype, B, M, N, L, k, V, T)
                ld = -(-N // 8) * 8
                assert need <= (M + B) * ld * size + (32 << 20) + 1024
