"""Limits of the attention over the paged cache: batches whose launches would not fit are refused
before anything reaches a GPU (no device work is issued by these tests)."""
import ctypes

import pytest

from trellis_coded_bit_amd import _lib

E = _lib
FAKE = 0x7F0000001000  # never dereferenced
FAR = 1 << 40


def _attend(heads, q_heads, seqs, rows):
    """The call without a workspace: TCQ_EWORKSPACE once it is found to fit."""
    cache = _lib.TcqCache(FAKE, FAKE + FAR, FAKE + 2 * FAR, FAKE + 3 * FAR, 10, heads, 16, 64,
                          E.TCQ_FP8)
    batch = _lib.TcqCacheBatch(FAKE + 4 * FAR, 5, 5, FAKE + 5 * FAR, FAKE + 6 * FAR, seqs)
    row = q_heads * 64
    return _lib.load().tcq_cache_attention(cache, batch, E.TCQ_BF16, FAKE + 7 * FAR, row, 64,
                                           q_heads, rows, 0.125, FAKE + 20 * FAR, row, 64, None, 0,
                                           None)


def _query(heads, q_heads, seqs, rows):
    b = ctypes.c_size_t(0)
    return _lib.load().tcq_cache_attention_workspace_bytes(64, heads, q_heads, seqs, rows,
                                                           ctypes.byref(b))


# (heads, q_heads, seqs, rows): the larger tiles' launch has 512 threads to a workgroup, of which
# 2^23 make 2^32
@pytest.mark.parametrize("call", [(8, 32, 1038576, 4180000), (8, 32, 1 << 20, (1 << 22) + 1),
                                  (9, 153, 900000, 900000), (16, 16, 523000, 8368100)])
def test_launches_that_do_not_fit(call):
    assert _attend(*call) == E.TCQ_EUNSUPPORTED
    assert _query(*call) == E.TCQ_EUNSUPPORTED


@pytest.mark.parametrize("call", [(8, 8, 1 << 20, 1 << 20),          # tiles of 16 rows alone
                                  (8, 32, 1 << 20, 1 << 20), (8, 32, 900000, 3700000),
                                  (16, 16, 450000, 7300000), (1, 1, 3, 1 << 23)])
def test_launches_that_fit(call):
    assert _attend(*call) == E.TCQ_EWORKSPACE
    assert _query(*call) == E.TCQ_OK
