"""Refusals of the norm, convolution and scan entry points that need no GPU: every status is decided on the host, before
a device is touched, and the Python surface raises ValueError for tensors that are not on a GPU."""

import ctypes

import pytest
import torch

from gated_delta_rule_38_gb300 import _lib
from gated_delta_rule_38_gb300 import build as gbuild
import gated_delta_rule_38_gb300 as gdr

P = 0x100000  # a made-up, aligned device address
SHAPE, DTYPE, NULL, UNSUPPORTED, ALIGN, WORKSPACE = 2, 3, 1, 4, 6, 7


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return _lib.load()


@pytest.fixture(autouse=True)
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("made-up device addresses are only passed on machines without a GPU")


def norm(**kw):
    p = _lib.NormProblem(7, 64, 64, 0, 2, 0, 0, 0, 1e-6)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def conv(**kw):
    p = _lib.ConvProblem(2, 5, 64, 4, 64, 0, 2, None, 0, 0)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def scan(**kw):
    p = _lib.ScanProblem(2, 5, 64, 16, 2, 64, 64, 64, 32, 32, 0, None, 0, 0)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def norm_fwd(lib, p, x=P, w=P, r=None, y=P, ro=None, s=None):
    return lib.gdr_norm_fwd(ctypes.byref(p), x, w, r, y, ro, s, None)


@pytest.mark.parametrize("kw,want", [
    (dict(D=0), SHAPE), (dict(D=16385, x_ld=16385), SHAPE), (dict(rows=-1), SHAPE), (dict(x_ld=63), SHAPE),
    (dict(scale_group=64), SHAPE), (dict(dtype=2), DTYPE), (dict(weight_dtype=1), DTYPE), (dict(residual_dtype=1), DTYPE),
    (dict(y_dtype=2), DTYPE)])
def test_norm_problem(lib, kw, want):
    assert norm_fwd(lib, norm(**kw)) == want
    n = ctypes.c_size_t()
    assert lib.gdr_norm_bwd_workspace_size(ctypes.byref(norm(**kw)), ctypes.byref(n)) == want


def test_norm_pointers(lib):
    p = norm()
    assert lib.gdr_norm_fwd(None, P, P, None, P, None, None, None) == NULL
    assert norm_fwd(lib, p, x=None) == NULL and norm_fwd(lib, p, w=None) == NULL and norm_fwd(lib, p, y=None) == NULL
    assert norm_fwd(lib, p, r=P) == NULL and norm_fwd(lib, p, ro=P) == NULL  # a residual and its output go together
    assert norm_fwd(lib, norm(y_dtype=3)) == NULL  # 8-bit output without scales
    assert norm_fwd(lib, p, x=P + 1) == ALIGN and norm_fwd(lib, p, w=P + 2) == ALIGN
    assert norm_fwd(lib, norm(rows=0), x=None, y=None) == 0
    n = ctypes.c_size_t()
    assert lib.gdr_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 0
    bwd = lambda ws, size, dres_in=None: lib.gdr_norm_bwd(ctypes.byref(p), P, P, P, None, P, dres_in, P, ws, size, None)  # noqa: E731
    assert bwd(None, 0) == WORKSPACE and bwd(P, n.value - 1) == WORKSPACE and bwd(P + 16, n.value) == ALIGN
    assert bwd(P, n.value, P) == DTYPE  # an fp32 gradient of a 16-bit residual stream


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), SHAPE), (dict(T=-1), SHAPE), (dict(D=0), SHAPE), (dict(W=1), SHAPE), (dict(W=5), SHAPE), (dict(x_ld=63), SHAPE),
    (dict(cu_seqlens=P, num_seqs=3), SHAPE), (dict(B=1, cu_seqlens=P, num_seqs=0), SHAPE), (dict(dtype=2), DTYPE),
    (dict(weight_dtype=1), DTYPE), (dict(flags=2), UNSUPPORTED)])
def test_conv_problem(lib, kw, want):
    p = conv(**kw)
    assert lib.gdr_conv_fwd(ctypes.byref(p), P, P, None, None, P, None, None) == want
    assert lib.gdr_conv_step(ctypes.byref(p), P, P, None, P, P, None) == want
    n = ctypes.c_size_t()
    assert lib.gdr_conv_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == want


def test_conv_pointers(lib):
    p = conv()
    fwd = lambda x=P, w=P, s=None, y=P, f=None: lib.gdr_conv_fwd(ctypes.byref(p), x, w, None, s, y, f, None)  # noqa: E731
    assert fwd(x=None) == NULL and fwd(w=None) == NULL and fwd(y=None) == NULL
    assert fwd(s=P, f=P) == UNSUPPORTED  # the states in place are the step's
    assert fwd(x=P + 1) == ALIGN and fwd(w=P + 2) == ALIGN
    assert lib.gdr_conv_step(ctypes.byref(p), P, P, None, None, P, None) == NULL
    packed = conv(B=1, cu_seqlens=P, num_seqs=3)
    assert lib.gdr_conv_step(ctypes.byref(packed), P, P, None, P, P, None) == UNSUPPORTED
    n = ctypes.c_size_t()
    assert lib.gdr_conv_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 0
    bwd = lambda ws, size, db=None: lib.gdr_conv_bwd(ctypes.byref(p), P, P, None, P, None, None, P, P, db, None, ws, size, None)  # noqa: E731
    assert bwd(None, 0) == WORKSPACE and bwd(P, n.value - 1) == WORKSPACE and bwd(P + 16, n.value) == ALIGN
    assert bwd(P, n.value, P) == NULL  # a bias gradient without a bias


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), SHAPE), (dict(T=-1), SHAPE), (dict(D=0), SHAPE), (dict(N=0), SHAPE), (dict(N=65), SHAPE), (dict(G=0), SHAPE),
    (dict(G=3), SHAPE), (dict(x_ld=63), SHAPE), (dict(dt_ld=1), SHAPE), (dict(z_ld=1), SHAPE), (dict(b_ld=31), SHAPE),
    (dict(c_ld=31), SHAPE), (dict(cu_seqlens=P, num_seqs=3), SHAPE), (dict(dtype=2), DTYPE), (dict(flags=2), UNSUPPORTED)])
def test_scan_problem(lib, kw, want):
    p = scan(**kw)
    n = ctypes.c_size_t()
    assert lib.gdr_scan_saved_bytes(ctypes.byref(p), ctypes.byref(n)) == want
    assert lib.gdr_scan_workspace_size(ctypes.byref(p), 1, ctypes.byref(n)) == want
    assert lib.gdr_scan_fwd(ctypes.byref(p), *[P] * 13, 1 << 40, None) == want
    assert lib.gdr_scan_step(ctypes.byref(p), *[P] * 10, None) == want
    assert lib.gdr_scan_bwd(ctypes.byref(p), *[P] * 22, 1 << 40, None) == want


def test_scan_pointers(lib):
    p, n = scan(), ctypes.c_size_t()
    fwd_names = ("x", "dt", "A", "B", "C", "D", "z", "bias", "s", "y", "f", "saved", "ws")

    def fwd(size=1 << 40, q=p, **kw):
        a = dict.fromkeys(fwd_names, P) | dict(D=None, z=None, bias=None, s=None, f=None, saved=None, ws=None) | kw
        return lib.gdr_scan_fwd(ctypes.byref(q), *[a[k] for k in fwd_names], size, None)

    for k in ("x", "dt", "A", "B", "C", "y"):
        assert fwd(**{k: None}) == NULL, k
    for k, off in (("x", 1), ("A", 2), ("B", 1), ("s", 2), ("saved", 8), ("D", 2)):
        assert fwd(**{k: P + off}) == ALIGN, k
    assert fwd(s=P, f=P) == UNSUPPORTED
    long = scan(B=1, T=4096)
    assert lib.gdr_scan_workspace_size(ctypes.byref(long), 0, ctypes.byref(n)) == 0 and n.value > 0
    assert fwd(q=long) == WORKSPACE and fwd(q=long, ws=P, size=n.value - 1) == WORKSPACE
    assert fwd(q=long, ws=P + 16, size=n.value) == ALIGN
    assert lib.gdr_scan_step(ctypes.byref(p), P, P, P, P, P, None, None, None, None, P, None) == NULL
    packed = scan(B=1, cu_seqlens=P, num_seqs=2)
    assert lib.gdr_scan_step(ctypes.byref(packed), *[P] * 10, None) == UNSUPPORTED
    names = ("x", "dt", "A", "B", "C", "D", "z", "bias", "dy", "s", "df", "saved", "dx", "ddt", "dA", "dB", "dC", "dD", "dz",
             "dbias", "ds", "ws")

    def bwd(size=1 << 40, **kw):
        a = dict.fromkeys(names, P) | kw
        return lib.gdr_scan_bwd(ctypes.byref(p), *[a[k] for k in names], size, None)

    for k in ("x", "dt", "A", "B", "C", "dy", "saved", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias"):
        assert bwd(**{k: None}) == NULL, k
    assert bwd(D=None) == NULL and bwd(z=None) == NULL and bwd(bias=None) == NULL  # gradients of what was not given
    assert bwd(ws=None) == WORKSPACE and bwd(size=0) == WORKSPACE and bwd(ws=P + 16) == ALIGN


def test_python_surface_needs_cuda_tensors():
    x, w = torch.zeros(1, 2, 8, dtype=torch.bfloat16), torch.zeros(8)
    for call in (lambda: gdr.rms_norm_fwd(x, w), lambda: gdr.rms_norm_bwd(x, w, x), lambda: gdr.rms_norm(x, w),
                 lambda: gdr.short_conv_fwd(x, torch.zeros(8, 4)), lambda: gdr.short_conv_step(x, x, torch.zeros(8, 4)),
                 lambda: gdr.selective_scan_fwd(x, x, torch.zeros(8, 4), x, x), lambda: gdr.rms_norm_fwd(None, w)):
        with pytest.raises(ValueError):
            call()
