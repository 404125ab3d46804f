"""What the norm, convolution and scan entry points refuse on the host: sizes that their kernels count in 32 bits, outputs
over inputs that other threads still read.  Needs no GPU."""

import ctypes

import pytest
import torch

from gated_delta_rule_38_gb300 import _lib
from gated_delta_rule_38_gb300 import build as gbuild

P = 0x100000  # a made-up, aligned device address
SHAPE, UNSUPPORTED = 2, 4


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return _lib.load()


@pytest.fixture
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("made-up device addresses are only passed on machines without a GPU")


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


# x: 10 tokens of 64 channels; y and the states [2,3,64] at these bytes from it
X, S = 10 * 64 * 2, 2 * 3 * 64 * 2


@pytest.mark.parametrize("y,ld,refused", [
    (0, 64, True), (2, 64, True), (-2, 64, True), (X - 2, 64, True), (2 - X, 64, True), (X, 64, False), (-X, 64, False),
    # rows 11 times as far apart: y fits between two of them, or touches the next one or the last
    (128, 704, False), (126, 704, True), (130, 704, True), (9 * 1408, 704, True), (9 * 1408 + 128, 704, False)])
def test_conv_output_over_tokens(lib, no_gpu, y, ld, refused):
    p = _lib.ConvProblem(2, 5, 64, 4, ld, 0, 2, None, 0, 0)
    far = P + (1 << 24)
    assert (lib.gdr_conv_fwd(ctypes.byref(p), P, far, None, None, P + y, None, None) == UNSUPPORTED) == refused
    w = far + (1 << 20)
    bwd = lambda x, dy, dx: lib.gdr_conv_bwd(ctypes.byref(p), x, far, None, dy, None, None, dx, far, None, None, w, 1 << 20, None)  # noqa: E731
    assert (bwd(P, far + 4096, P + y) == UNSUPPORTED) == refused
    if ld == 64:
        assert (bwd(far + 4096, P, P + y) == UNSUPPORTED) == refused
    # the step's threads read and write a token each on their own
    assert lib.gdr_conv_step(ctypes.byref(p), P, far, None, far, P + y, None) != UNSUPPORTED


@pytest.mark.parametrize("at,refused", [(0, True), (2, True), (S - 2, True), (-2, True), (S, False), (-S, False)])
def test_conv_states_over_states(lib, no_gpu, at, refused):
    p = _lib.ConvProblem(2, 5, 64, 4, 64, 0, 2, None, 0, 0)
    far = P + (1 << 24)
    fwd = lambda y, f, x=far + 4096: lib.gdr_conv_fwd(ctypes.byref(p), x, far, None, P, y, f, None)  # noqa: E731
    assert (fwd(far + 8192, P + at) == UNSUPPORTED) == refused
    assert (fwd(P + at, None) == UNSUPPORTED) == (refused or at == -S)  # (y is longer than the states)
    assert fwd(far + 8192, far + 4096 + 64) == UNSUPPORTED  # over the tokens
    bwd = lambda s, ds, out: lib.gdr_conv_bwd(ctypes.byref(p), far + 4096, far, None, far + 8192, s, ds, far + 16384, far, None, out,  # noqa: E731
                                              far + (1 << 20), 1 << 20, None)
    assert (bwd(P, None, P + at) == UNSUPPORTED) == refused and (bwd(None, P, P + at) == UNSUPPORTED) == refused
