"""Refusals of linear attention, the gated norm and the block norm that need no GPU: decided on the host, before a device is
touched; and the sizes of workspaces."""

import ctypes

import pytest
import torch

from gated_delta_rule_38_gb300 import _lib
from gated_delta_rule_38_gb300 import build as gbuild
import gated_delta_rule_38_gb300 as gdr

P = 0x10000000  # a made-up, aligned device address; tensors FAR apart do not touch
FAR = 1 << 34
NULL, SHAPE, DTYPE, UNSUPPORTED, ALIGN, WORKSPACE = 1, 2, 3, 4, 6, 7


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return _lib.load()


@pytest.fixture(autouse=True)
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("made-up device addresses are only passed on machines without a GPU")


def far(names, given=()):
    return {n: P + (i + 1) * FAR for i, n in enumerate(names)} | dict(given)


def lin(**kw):
    p = _lib.LinProblem(2, 300, 2, 4, 64, 96, 128, 128, 384, 0, 0.125, None, 0)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


FWD = ("q", "k", "v", "decay", "s", "o", "f", "ws")
BWD = ("q", "k", "v", "decay", "do", "s", "df", "dq", "dk", "dv", "ds", "ws")


def fwd(lib, p, size=1 << 40, **kw):
    a = far(FWD, kw)
    return lib.gdr_lin_fwd(ctypes.byref(p), *[a[n] for n in FWD], size, None)


def bwd(lib, p, size=1 << 40, **kw):
    a = far(BWD, kw)
    return lib.gdr_lin_bwd(ctypes.byref(p), *[a[n] for n in BWD], size, None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), SHAPE), (dict(T=-1), SHAPE), (dict(Hk=0), SHAPE), (dict(H=0), SHAPE), (dict(H=3), SHAPE), (dict(K=0), SHAPE), (dict(K=60), SHAPE),
    (dict(K=136), SHAPE), (dict(V=4), SHAPE), (dict(V=129), SHAPE), (dict(q_ld=127), SHAPE), (dict(k_ld=127), SHAPE), (dict(v_ld=383), SHAPE),
    (dict(cu_seqlens=P, num_seqs=3), SHAPE), (dict(B=1, cu_seqlens=P, num_seqs=0), SHAPE), (dict(B=1 << 20, T=1 << 11), SHAPE),
    (dict(B=1 << 29, T=2, H=128, Hk=128, q_ld=1 << 20, k_ld=1 << 20, v_ld=1 << 20), SHAPE), (dict(dtype=2), DTYPE)])
def test_lin_problem(lib, kw, want):
    p = lin(**kw)
    n = ctypes.c_size_t()
    assert lib.gdr_lin_workspace_size(ctypes.byref(p), 0, ctypes.byref(n)) == want
    assert fwd(lib, p) == want and bwd(lib, p) == want
    assert lib.gdr_lin_step(ctypes.byref(p), *[P + i * FAR for i in range(6)], None) == want


def test_lin_pointers(lib):
    p = lin()
    assert lib.gdr_lin_workspace_size(None, 0, None) == NULL and lib.gdr_lin_workspace_size(ctypes.byref(p), 0, None) == NULL
    for n in ("q", "k", "v", "decay", "o"):
        assert fwd(lib, p, **{n: None}) == NULL, n
    for n, off in (("q", 2), ("k", 8), ("v", 8), ("decay", 2), ("s", 4), ("o", 8), ("f", 4)):
        assert fwd(lib, p, **{n: P + off}) == ALIGN, n
    assert fwd(lib, lin(q_ld=132)) == ALIGN and fwd(lib, lin(v_ld=385)) == ALIGN
    q, v = P + FAR, P + 3 * FAR
    assert fwd(lib, p, s=P, f=P) == UNSUPPORTED and fwd(lib, p, s=P, f=P + 2 * 4 * 64 * 96 * 4 - 16) == UNSUPPORTED
    assert fwd(lib, p, o=v) == UNSUPPORTED and fwd(lib, p, o=q) == UNSUPPORTED
    for n in ("q", "k", "v", "decay", "do", "dq", "dk", "dv"):
        assert bwd(lib, p, **{n: None}) == NULL, n
    for n in ("dq", "dk", "dv"):
        assert bwd(lib, p, **{n: v}) == UNSUPPORTED and bwd(lib, p, **{n: q}) == UNSUPPORTED, n
    assert bwd(lib, p, df=P, ds=P) == UNSUPPORTED and bwd(lib, p, s=P, ds=P) == UNSUPPORTED
    step = lambda q=P, k=P + FAR, v=P + 2 * FAR, d=P + 3 * FAR, s=P + 4 * FAR, o=P + 5 * FAR, pp=p: lib.gdr_lin_step(  # noqa: E731
        ctypes.byref(pp), q, k, v, d, s, o, None)
    assert step(q=None) == NULL and step(s=None) == NULL and step(q=P + 1) == ALIGN and step(s=P + 4 * FAR + 8) == ALIGN
    assert step(o=P) == UNSUPPORTED and step(pp=lin(B=1, cu_seqlens=P, num_seqs=2)) == UNSUPPORTED
    assert step(pp=lin(T=0), q=None) == 0


def test_lin_outputs_over_states_and_one_another(lib):
    p, sb = lin(), 2 * 4 * 64 * 96 * 4
    a = far(FWD)
    assert fwd(lib, p, o=a["s"]) == UNSUPPORTED and fwd(lib, p, o=a["f"] + sb - 16) == UNSUPPORTED and fwd(lib, p, f=a["o"] + 16) == UNSUPPORTED
    a = far(BWD)
    for n in ("dq", "dk", "dv"):
        for m in ("s", "df", "ds"):
            assert bwd(lib, p, **{n: a[m] + sb - 16}) == UNSUPPORTED and bwd(lib, p, **{m: a[n] + 16}) == UNSUPPORTED, (n, m)
        for m in {"dq", "dk", "dv"} - {n}:
            assert bwd(lib, p, **{n: a[m] + 16}) == UNSUPPORTED, (n, m)
    s = P + 4 * FAR
    assert lib.gdr_lin_step(ctypes.byref(p), P, P + FAR, P + 2 * FAR, P + 3 * FAR, s, s + 32, None) == UNSUPPORTED


def test_lin_workspaces(lib):
    n = ctypes.c_size_t()

    def size(p, backward):
        assert lib.gdr_lin_workspace_size(ctypes.byref(p), backward, ctypes.byref(n)) == 0
        return n.value

    assert size(lin(T=100, Hk=4, q_ld=256, k_ld=256), 0) == 0  # one chunk a row: nothing to cut, nothing to share
    assert size(lin(T=100), 1) == 2 * 2 * 100 * 4 * 64 * 4  # fp32 dq and dk of every head
    long = lin(B=1, T=1 << 17)
    need = size(long, 0)
    assert 0 < need < 1 << 30
    assert fwd(lib, long, ws=None) == WORKSPACE and fwd(lib, long, need - 1) == WORKSPACE and fwd(lib, long, need, ws=P + 16) == ALIGN
    need = size(long, 1)
    assert bwd(lib, long, ws=None) == WORKSPACE and bwd(lib, long, need - 1) == WORKSPACE and bwd(lib, long, need, ws=P + 16) == ALIGN


def test_lin_workspace_of_many_sequences(lib):
    """The states that segments exchange are those of intervals of the token axis, of the heads' own size, however many sequences
    a packed batch has; and a batch of many short ones is not cut."""
    n = ctypes.c_size_t()

    def size(T, N, H=32, K=128, V=128, backward=0):
        p = _lib.LinProblem(1, T, H, H, K, V, H * K, H * K, H * V, 0, 1.0, P, N)
        assert lib.gdr_lin_workspace_size(ctypes.byref(p), backward, ctypes.byref(n)) == 0
        return n.value

    for T, H in ((16384, 32), (8192, 32), (65536, 4), (3000, 2)):
        for N in (2, 7, 64, 1024, 4096):
            for b in (0, 1):
                # at most a state of 64 KB of every chunk, head and walk (q, k, v and o: 128 KB)
                assert size(T, N, H, backward=b) <= (1 + b) * (T // 128 + 1) * H * 65536, (T, H, N, b)
    assert size(65536, 3, 4) > 0 and size(65536, 3, 4, 32, 64) <= size(65536, 3, 4) // 8 + 512
    for T, N in ((16384, 1024), (8192, 4096)):
        assert size(T, N) == 0 and size(T, N, backward=1) == 0


def gated(**kw):
    p = _lib.GatedNormProblem(7, 256, 256, 4, 64, 0, 2, 2, 1e-6)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def block(**kw):
    p = _lib.BlockNormProblem(7, 64, 64, 64, 0, 2, 2, 1, 0.5, 1e-6)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


G_FWD, G_BWD = ("x", "g", "w", "y"), ("x", "g", "w", "dy", "dx", "dg", "dw", "ws")
B_FWD, B_BWD = ("x", "r", "w", "pw", "g", "y", "h"), ("x", "h", "w", "pw", "g", "dy", "dr", "dx", "dri", "dw", "dpw", "dg", "ws")


def call(fn, names, p, size=None, **kw):
    a = far(names, kw)
    return fn(ctypes.byref(p), *[a[n] for n in names], *(() if size is None else (size,)), None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), SHAPE), (dict(heads=0), SHAPE), (dict(D=0), SHAPE), (dict(D=16385, x_ld=1 << 20, gate_ld=1 << 20), SHAPE),
    (dict(D=16377, x_ld=1 << 20, gate_ld=1 << 20), SHAPE), (dict(x_ld=255), SHAPE), (dict(gate_ld=255), SHAPE), (dict(tokens=1 << 40), SHAPE),
    (dict(dtype=2), DTYPE), (dict(weight_dtype=1), DTYPE), (dict(gate_act=0), UNSUPPORTED), (dict(gate_act=3), UNSUPPORTED)])
def test_gated_problem(lib, kw, want):
    p, n = gated(**kw), ctypes.c_size_t()
    assert call(lib.gdr_gated_norm_fwd, G_FWD, p) == want and call(lib.gdr_gated_norm_bwd, G_BWD, p, 1 << 40) == want
    assert lib.gdr_gated_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), SHAPE), (dict(D=0), SHAPE), (dict(D=16385, x_ld=1 << 20, gate_ld=1 << 20), SHAPE), (dict(x_ld=63), SHAPE), (dict(gate_ld=63), SHAPE),
    (dict(D=16383, x_ld=16383, gate_ld=16383), SHAPE), (dict(dtype=2), DTYPE), (dict(weight_dtype=1), DTYPE), (dict(residual_dtype=1), DTYPE),
    (dict(gate_act=3), UNSUPPORTED)])
def test_block_problem(lib, kw, want):
    p, n = block(**kw), ctypes.c_size_t()
    assert call(lib.gdr_block_norm_fwd, B_FWD, p) == want and call(lib.gdr_block_norm_bwd, B_BWD, p, 1 << 40) == want
    assert lib.gdr_block_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == want


def test_norm_pointers(lib):
    p, b, n = gated(), block(), ctypes.c_size_t()
    for k in G_FWD:
        assert call(lib.gdr_gated_norm_fwd, G_FWD, p, **{k: None}) == NULL, k
        assert call(lib.gdr_gated_norm_fwd, G_FWD, p, **{k: P + 8}) == ALIGN, k
    assert call(lib.gdr_gated_norm_fwd, G_FWD, p, y=P + FAR) == UNSUPPORTED and call(lib.gdr_gated_norm_fwd, G_FWD, p, y=P + 2 * FAR) == UNSUPPORTED
    assert call(lib.gdr_gated_norm_fwd, G_FWD, gated(x_ld=260)) == ALIGN  # rows of whole vectors,
    assert call(lib.gdr_gated_norm_fwd, G_FWD, gated(D=63)) == ALIGN      # or tensors without gaps
    assert call(lib.gdr_gated_norm_fwd, G_FWD, gated(tokens=0), x=None) == 0
    assert lib.gdr_gated_norm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 0
    g = lib.gdr_gated_norm_bwd
    for k in G_BWD[:-1]:
        assert call(g, G_BWD, p, n.value, **{k: None}) == NULL, k
    assert call(g, G_BWD, p, n.value, ws=None) == WORKSPACE and call(g, G_BWD, p, n.value - 1) == WORKSPACE and call(g, G_BWD, p, n.value, ws=P + 16) == ALIGN
    assert call(g, G_BWD, p, n.value, dx=P + FAR) == UNSUPPORTED and call(g, G_BWD, p, n.value, dg=P + 4 * FAR) == UNSUPPORTED
    f = lib.gdr_block_norm_fwd
    for k in ("x", "r", "w", "y", "h"):
        assert call(f, B_FWD, b, **{k: None}) == NULL, k
    for k in B_FWD:
        assert call(f, B_FWD, b, **{k: P + 8}) == ALIGN, k
    a = far(B_FWD)
    assert call(f, B_FWD, b, y=a["x"]) == UNSUPPORTED and call(f, B_FWD, b, y=a["h"]) == UNSUPPORTED and call(f, B_FWD, b, y=a["r"]) == UNSUPPORTED
    assert call(f, B_FWD, b, h=a["r"] + 32) == UNSUPPORTED and call(f, B_FWD, b, h=a["g"]) == UNSUPPORTED
    assert call(f, B_FWD, block(gate_ld=68)) == ALIGN and call(f, B_FWD, block(rows=0), x=None) == 0
    assert lib.gdr_block_norm_bwd_workspace_size(ctypes.byref(b), ctypes.byref(n)) == 0 and n.value > 0
    g = lib.gdr_block_norm_bwd
    for k in ("x", "h", "w", "dy", "dx", "dri", "dw"):
        assert call(g, B_BWD, b, n.value, **{k: None}) == NULL, k
    for k in ("pw", "dpw", "g", "dg"):  # a weight or gate and its gradient go together
        assert call(g, B_BWD, b, n.value, **{k: None}) == NULL, k
    a = far(B_BWD)
    for k in ("dx", "dri", "dg"):
        for i in ("x", "h", "g", "dy", "dr"):
            assert call(g, B_BWD, b, n.value, **{k: a[i]}) == UNSUPPORTED, (k, i)
    assert call(g, B_BWD, b, n.value, ws=None) == WORKSPACE and call(g, B_BWD, b, n.value, ws=P + 16) == ALIGN


def test_norm_gradients_over_one_another(lib):
    a, g = far(G_BWD), lib.gdr_gated_norm_bwd
    p = gated()
    assert call(g, G_BWD, p, 1 << 40, dx=a["dg"] + 16) == UNSUPPORTED and call(g, G_BWD, p, 1 << 40, dg=a["dx"] + 16) == UNSUPPORTED
    a, g = far(B_BWD), lib.gdr_block_norm_bwd
    for n in ("dx", "dri", "dg"):
        for m in {"dx", "dri", "dg"} - {n}:
            assert call(g, B_BWD, block(), 1 << 40, **{n: a[m] + 16}) == UNSUPPORTED, (n, m)


def test_python_surface_needs_cuda_tensors():
    x, w = torch.zeros(1, 2, 1, 8, dtype=torch.bfloat16), torch.zeros(8)
    d = torch.zeros(1)
    for f in (lambda: gdr.linear_attention_fwd(x, x, x, d), lambda: gdr.linear_attention(x, x, x, d), lambda: gdr.linear_attention_step(x, x, x, d, x),
              lambda: gdr.linear_attention_bwd(x, x, x, d, x), lambda: gdr.linear_attention(x, x, x, d.requires_grad_()),
              lambda: gdr.gated_rms_norm_fwd(x, x, w), lambda: gdr.gated_rms_norm(x, x, w), lambda: gdr.gated_rms_norm_bwd(x, x, w, x),
              lambda: gdr.block_norm_fwd(x, x, w), lambda: gdr.block_norm(x, x, w), lambda: gdr.block_norm_bwd(x, x, w, x), lambda: gdr.block_norm_fwd(None, x, w)):
        with pytest.raises(ValueError):
            f()


def test_outputs_over_small_inputs(lib):
    """Decays, offsets and weights are inputs too, and states and weights' gradients outputs, as far as the last of their bytes."""
    cu, nb = P + 40 * FAR, 4  # offsets of three sequences, decays of four heads
    p, sb = lin(B=1, T=600, cu_seqlens=cu, num_seqs=3), 3 * 4 * 64 * 96 * 4
    a = far(FWD)
    last = dict(q=(599 * 128 + 127) * 2, k=(599 * 128 + 127) * 2, v=(599 * 384 + 383) * 2, decay=nb * 4 - 4, s=sb - 4)
    for n in ("o", "f"):
        for m, off in last.items():
            assert fwd(lib, p, **{n: (a[m] + off) // 16 * 16}) == UNSUPPORTED, (n, m)
        assert fwd(lib, p, **{n: cu}) == UNSUPPORTED, n
    a = far(BWD)
    last = dict(last, do=(600 * 384 - 1) * 2, df=sb - 4)
    for n in ("dq", "dk", "dv", "ds"):
        for m, off in last.items():
            assert bwd(lib, p, **{n: (a[m] + off) // 16 * 16}) == UNSUPPORTED, (n, m)
        assert bwd(lib, p, **{n: cu}) == UNSUPPORTED, n
        for m in {"dq", "dk", "dv", "ds"} - {n}:
            assert bwd(lib, p, **{n: a[m]}) == UNSUPPORTED, (n, m)
    p = lin()
    step = ("q", "k", "v", "decay", "s", "o")
    a = far(step)
    for n in ("o", "s"):
        for m in ("q", "k", "v", "decay"):
            assert call(lib.gdr_lin_step, step, p, **{n: a[m]}) == UNSUPPORTED, (n, m)
    a, p = far(G_FWD), gated()
    assert call(lib.gdr_gated_norm_fwd, G_FWD, p, y=a["w"] + 64 * 4 - 16) == UNSUPPORTED
    a = far(G_BWD)
    for n in ("dx", "dg", "dw"):
        for m in {"x", "g", "w", "dy", "dx", "dg", "dw"} - {n}:
            assert call(lib.gdr_gated_norm_bwd, G_BWD, p, 1 << 40, **{n: a[m]}) == UNSUPPORTED, (n, m)
    a, p = far(B_FWD), block()
    for n in ("y", "h"):
        for m in ("w", "pw"):
            assert call(lib.gdr_block_norm_fwd, B_FWD, p, **{n: a[m] + 64 * 4 - 16}) == UNSUPPORTED, (n, m)
    a = far(B_BWD)
    outs = ("dx", "dri", "dw", "dpw", "dg")
    for n in outs:
        for m in {"x", "h", "w", "pw", "g", "dy", "dr", *outs} - {n}:
            assert call(lib.gdr_block_norm_bwd, B_BWD, p, 1 << 40, **{n: a[m]}) == UNSUPPORTED, (n, m)
    # without a gate or a post_weight their addresses are nobody's
    none = dict(g=None, dg=None, pw=None, dpw=None)
    assert call(lib.gdr_block_norm_bwd, B_BWD, p, 1 << 40, dw=a["dpw"], **none) != UNSUPPORTED


@pytest.mark.parametrize("D", [8193, 9001, 10191, 10201, 12288, 16375, 16384])
def test_partial_rows_are_as_many_as_fit(lib, D):
    """Four vectors a thread, one block an SM: no more blocks leave partial rows than run at once."""
    n = ctypes.c_size_t()
    assert lib.gdr_gated_norm_bwd_workspace_size(ctypes.byref(gated(tokens=100000, heads=1, D=D, x_ld=D, gate_ld=D)), ctypes.byref(n)) == 0
    assert n.value <= 152 * D * 4 + 255
    assert lib.gdr_block_norm_bwd_workspace_size(ctypes.byref(block(rows=100000, D=D, x_ld=D, gate_ld=D)), ctypes.byref(n)) == 0
    assert n.value <= 2 * 152 * D * 4 + 255
