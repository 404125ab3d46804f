"""Sizes that the norm, convolution and scan entry points refuse on the host because their kernels count in 32 bits.
Needs no GPU."""

import ctypes

import pytest

from gated_delta_rule_38_gb300 import _lib
from gated_delta_rule_38_gb300 import build as gbuild

SHAPE = 2


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return _lib.load()


def scan_saved(lib, B, T, D, N, G):
    p, n = _lib.ScanProblem(B, T, D, N, G, D, D, D, G * N, G * N, 0, None, 0, 0), ctypes.c_size_t()
    return lib.gdr_scan_saved_bytes(ctypes.byref(p), ctypes.byref(n)), n.value


@pytest.mark.parametrize("N,pad", [(1, 512), (4, 512), (5, 256), (16, 128)])
def test_scan_padded_channels(lib, N, pad):
    """A group's channels are padded to a block's: as many groups of one channel as 31 bits hold, and one more power of two."""
    G = (1 << 31) // pad // 2
    states = 4 * max(1, 1 << (N - 1).bit_length() >> 2)
    assert scan_saved(lib, 1, 1, G, N, G) == (0, G * pad * states * 4)
    assert scan_saved(lib, 1, 1, 2 * G, N, 2 * G)[0] == SHAPE


def test_scan_rows(lib):
    assert scan_saved(lib, 1 << 30, 1, 1, 1, 1)[0] == 0
    assert scan_saved(lib, (1 << 30) + 1, 1, 1, 1, 1)[0] == SHAPE
