"""Workspace sizes of the attention over the paged cache and of the microscaled layer: one that
serves a batch serves every smaller one (the queries touch no GPU)."""
import numpy as np
import pytest

from trellis_coded_bit_amd import _lib


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,q_heads", [(1, 1), (8, 8), (8, 32), (2, 34), (1, 128)])
def test_attention_need_grows_with_the_batch(heads, q_heads, dim):
    def need(seqs, rows):
        return _lib.tcq_cache_attention_workspace_bytes(dim, heads, q_heads, seqs, rows)

    rng = np.random.default_rng(heads * q_heads)
    seqs = sorted({1, 2, 3, 15, 16, 17, 63, 64, 65, 66, 67, 68, 69, 128, 1000, 4096, 1 << 16,
                   *(int(s) for s in np.exp(rng.uniform(0, 11, 20)))})
    rows = sorted({1, 2, 3, 15, 16, 17, 63, 64, 65, 1023, 1024, 4096, 1 << 16,
                   *(int(r) for r in np.exp(rng.uniform(0, 11, 20)))})
    table = [[need(s, r) for r in rows] for s in seqs]
    for a in table:
        assert a == sorted(a)
    for a in zip(*table):
        assert list(a) == sorted(a)


def test_attention_need_stays_near_the_shares():
    """2048 shares of 16 rows and 512 of 256, whose rows hold the outputs, a maximum and a sum, and
    24 bytes a sequence."""
    for dim in (64, 128, 256):
        for seqs, rows in ((1, 1), (64, 64), (1 << 16, 1 << 16), (4, 8192)):
            need = _lib.tcq_cache_attention_workspace_bytes(dim, 8, 32, seqs, rows)
            assert need <= (2048 * 16 + 512 * 256) * (dim + 2) * 4 + 24 * seqs + 1024


SHAPES = [(4096, 4096), (14336, 4096), (4096, 14336), (2048, 2048), (64, 512), (130, 153), (1, 64),
          (1031, 4160), (300, 500), (16, 1 << 17), (1, 1), (7000, 6200)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("fmt", [_lib.TCQ_FP4, _lib.TCQ_FP8])
def test_layer_need_grows_with_the_batch(shape, fmt):
    rng = np.random.default_rng(sum(shape))
    batches = sorted({*range(0, 530), 1023, 1024, 1025, 2048, 4096, 8192, 16384,
                      *(int(b) for b in np.exp(rng.uniform(5, 11, 300)))})
    need = [_lib.tcq_mx_linear_workspace_bytes(fmt, B, *shape) for B in batches]
    assert need == sorted(need)
    for dtype in (_lib.TCQ_F32, _lib.TCQ_F16, _lib.TCQ_BF16):
        for wanted in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)):
            need = [_lib.tcq_mx_linear_backward_workspace_bytes(dtype, B, *shape, *wanted)
                    for B in batches]
            assert need == sorted(need), (dtype, wanted)
