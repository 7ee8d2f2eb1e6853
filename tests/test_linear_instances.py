"""The library holds no kernel of the coded linear layer that no call reaches: the instances in
libtcq.so against the ways that the dispatch rules leave."""
import re
import shutil
import subprocess

import pytest

from trellis_coded_bit_amd import _lib, build

SIXTEEN = {"DF16_", "DF16b"}


def _instances(kernel):
    if not shutil.which("nm"):
        pytest.skip("nm is not here")
    _lib.load()
    names = subprocess.run(["nm", build.LIB], capture_output=True, text=True, check=True).stdout
    found = set()
    for m in re.finditer(r"_ZN3tcq12_GLOBAL__N_1\d+(?:__device_stub__)?" + kernel +
                         r"I(f|DF16_|DF16b)((?:L[ib]\d+E)+)E", names):
        found.add((m.group(1), *(int(v) for v in re.findall(r"L[ib](\d+)E", m.group(2)))))
    assert found
    return found


def test_small_kernels():
    """16-bit tables of several parts (V > 1) go up to 64 rows, 4 batch tiles; those of V = 1 are
    always one part."""
    for t, kv, V, bt, one in _instances("small_kernel"):
        assert kv % V == 0 and kv <= 4
        if t in SIXTEEN and not one:
            assert V > 1 and bt <= 4, (t, kv, V, bt, one)


def test_slope_kernels():
    """Two terms for 16-bit types alone; one term of theirs for none and relu (0, 1) alone."""
    for t, act, terms in _instances("slope_kernel"):
        assert terms == 1 if t == "f" else terms == 2 or act <= 1, (t, act, terms)
