"""The operators around the recurrence in a layer: RMS norm with the residual's addition (and an 8-bit output with
scales), the norm of a mixer's output with its gate, the norms behind and before a block around the residual's addition,
the short causal convolution, and the selective state space scan.

Python surface of ``gdr_norm_*``, ``gdr_gated_norm_*``, ``gdr_block_norm_*``, ``gdr_conv_*`` and ``gdr_scan_*`` in
``include/gdr.h``.  As for the delta rule, the ``*_fwd`` / ``*_bwd`` / ``*_step`` functions map onto one library call each
and ``rms_norm``, ``gated_rms_norm``, ``block_norm``, ``short_conv`` and ``selective_scan`` are differentiable (once: second
derivatives are refused).  Token tensors may be row-strided views (slices of a fused projection are read in place); any
other view is copied.
"""

from __future__ import annotations

from ctypes import byref, c_size_t
from functools import wraps

import torch

from . import _lib
from ._args import _DT, _check, _check_cu, _cu, _need, _row_stride, _rows

__all__ = ["rms_norm", "rms_norm_fwd", "rms_norm_bwd", "short_conv", "short_conv_fwd", "short_conv_bwd",
           "short_conv_step", "selective_scan", "selective_scan_fwd", "selective_scan_bwd", "selective_scan_step",
           "gated_rms_norm", "gated_rms_norm_fwd", "gated_rms_norm_bwd", "block_norm", "block_norm_fwd", "block_norm_bwd"]


def _p(t):
    return None if t is None else t.data_ptr()


def _s(t):
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _dt(t, name, allowed):
    if not isinstance(t, torch.Tensor):
        _check(t, name)
    if t.dtype not in allowed:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {', '.join(str(d) for d in allowed)}")
    return _DT[t.dtype]


_HALF = (torch.bfloat16, torch.float16)


def _tokens(x, name):
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype in _HALF):
        _check(x, name, contiguous=False)
        _dt(x, name, _HALF)
    return _DT[x.dtype]


def _workspace(fn, p, like):
    n = c_size_t(0)
    _lib.check(fn(byref(p), byref(n)), fn.__name__)
    return torch.empty(n.value, dtype=torch.uint8, device=like.device), n.value


class _Once(torch.autograd.Function):
    """Hands on the gradients that a backward pass computed, as depending on all that it read: who differentiates them is
    told, where torch's once_differentiable lets autograd.grad take the other terms of a loss alone."""

    @staticmethod
    def forward(ctx, name, grads, *read):
        ctx.name = name
        return tuple(None if g is None else g.detach() for g in grads)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.name} has no second derivatives")


def _once(backward):
    """A Function's backward that is not differentiable itself."""
    name = backward.__qualname__.split(".")[0].lstrip("_")

    @wraps(backward)
    def run(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():  # (no graph of the backward pass was asked for)
            return out
        return _Once.apply(name, out, *ctx.saved_tensors, *grads)

    return run


# ---------------------------------------------------------------- RMS norm

def rms_norm_fwd(x, weight, residual=None, eps=1e-6, quant=None, scale_group=0, out=None):
    """(y, residual_out, scale): y = h / sqrt(mean(h^2) + eps) * weight with h = x + residual over the last dimension.

    x [..., D] bf16 or fp16; weight [D] of x's type or fp32; residual [..., D] of x's type or fp32 (the residual
    stream's type): residual_out is h in that type, None without a residual.  ``quant="e4m3"``: y is float8_e4m3fn
    holding y / scale, with scale fp32 [..., 1] per row (``scale_group=0``) or [..., ceil(D/128)] per 128 columns
    (``scale_group=128``); else scale is None.
    """
    xd = _tokens(x, "x")
    D = x.shape[-1]
    wd = _dt(weight, "weight", (x.dtype, torch.float32))
    _need(weight, "weight", (D,), weight.dtype, x)
    rd = xd
    if residual is not None:
        rd = _dt(residual, "residual", (x.dtype, torch.float32))
        _need(residual, "residual", x.shape, residual.dtype, x)
    if quant not in (None, "e4m3"):
        raise ValueError(f"quant is {quant!r}, expected None or 'e4m3'")
    if scale_group not in (0, 128):
        raise ValueError(f"scale_group is {scale_group}, expected 0 or 128")
    x, ld = _rows(x)
    if D % 8 == 0 and (ld % 8 or x.data_ptr() % 16):  # a copy takes the whole-vector form, whose bits are those of any
        x, ld = x.contiguous(), D                     # other view's
    yt = torch.float8_e4m3fn if quant else x.dtype
    if out is not None:
        _need(out, "out", x.shape, yt, x)
    y = out if out is not None else torch.empty(x.shape, dtype=yt, device=x.device)
    res_out = None if residual is None else torch.empty_like(residual)
    scale = None
    if quant:
        n = (D + 127) // 128 if scale_group else 1
        scale = torch.empty(x.shape[:-1] + (n,), dtype=torch.float32, device=x.device)
    p = _lib.NormProblem(x.numel() // D if D else 0, ld, D, xd, wd, rd, _lib.GDR_E4M3 if quant else xd, scale_group, eps)
    _lib.check(_lib.load().gdr_norm_fwd(byref(p), _p(x), _p(weight), _p(residual), _p(y), _p(res_out), _p(scale), _s(x)),
               "gdr_norm_fwd")
    return y, res_out, scale


def rms_norm_bwd(h, weight, dy, dresidual=None, eps=1e-6, dtype=None):
    """(dx, dresidual_in, dweight) at h, the forward's residual_out (or its x without a residual).

    dy [..., D] bf16 or fp16; ``dresidual`` (h's type) is the gradient that reaches residual_out from later layers.
    dx has dy's type (``dtype``, if given, must be it).  The residual's gradient equals dx: dresidual_in is None when
    h has that type too, and its fp32 form when h is fp32.
    """
    yd = _tokens(dy, "dy")
    hd = _dt(h, "h", (dy.dtype, torch.float32))
    _need(h, "h", dy.shape, h.dtype, dy, contiguous=False)
    if dtype is not None and dtype != dy.dtype:
        raise ValueError(f"dtype is {dtype}, dy has {dy.dtype}")
    D = h.shape[-1]
    wd = _dt(weight, "weight", (dy.dtype, torch.float32))
    _need(weight, "weight", (D,), weight.dtype, h)
    if dresidual is not None:
        _need(dresidual, "dresidual", h.shape, h.dtype, h)
    h, ld = _rows(h)
    dy = dy.contiguous()
    dx = torch.empty_like(dy)
    dres = torch.empty(h.shape, dtype=torch.float32, device=h.device) if hd == _lib.GDR_FP32 else None
    dw = torch.empty_like(weight)
    p = _lib.NormProblem(h.numel() // D if D else 0, ld, D, yd, wd, hd, yd, 0, eps)
    lib = _lib.load()
    ws, n = _workspace(lib.gdr_norm_bwd_workspace_size, p, h)
    _lib.check(lib.gdr_norm_bwd(byref(p), _p(h), _p(weight), _p(dy), _p(dresidual), _p(dx), _p(dres), _p(dw), _p(ws), n,
                                _s(h)), "gdr_norm_bwd")
    return dx, dres, dw


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, _ = rms_norm_fwd(x, weight, residual, eps)
        ctx.save_for_backward(x if h is None else h, weight)
        ctx.eps, ctx.dtype, ctx.has_res = eps, x.dtype, residual is not None
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @_once
    def backward(ctx, dy, dh):
        h, weight = ctx.saved_tensors
        if dy is None and dh is None:
            return None, None, None, None
        if dy is None:
            dy = torch.zeros(h.shape, dtype=ctx.dtype, device=h.device)
        dx, dres, dw = rms_norm_bwd(h, weight, dy, None if dh is None else dh.contiguous(), ctx.eps)
        return dx, dw, (dx if dres is None else dres) if ctx.has_res else None, None


def rms_norm(x, weight, residual=None, eps=1e-6):
    """Differentiable: (y, residual_out or None).  See rms_norm_fwd."""
    return _RmsNorm.apply(x, weight, None if residual is None else residual.contiguous(), eps)


# ---------------------------------------------------------------- norm of a mixer's output with its gate

_ACT = {None: _lib.GDR_GATE_RAW, "sigmoid": _lib.GDR_GATE_SIGMOID, "silu": _lib.GDR_GATE_SILU}


def _vectors(t, D, wide, inner):
    """(t, row stride) as the gated and the block norm read it: rows on 16-byte boundaries, or no gaps between them."""
    if t.is_contiguous():
        if t.data_ptr() % 16 == 0:
            return t, wide
        ld = wide
    else:
        t, ld = _rows(t, inner)
    if t.data_ptr() % 16 or (ld % 8 if D % 8 == 0 else ld != wide):
        return t.clone(memory_format=torch.contiguous_format), wide
    return t, ld


def _on16(t):
    """t on a 16-byte boundary, copied there if need be (a slice of a gradient or of a flat parameter may lie anywhere)."""
    if t is None or t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _gated_problem(x, gate, weight, eps, activation):
    xd = _tokens(x, "x")
    if x.dim() < 1:
        raise ValueError("x must be [..., D]")
    D = x.shape[-1]
    _need(gate, "gate", x.shape, x.dtype, x, False)
    wd = _dt(weight, "weight", (x.dtype, torch.float32))
    _need(weight, "weight", (D,), weight.dtype, x)
    if activation not in ("silu", "sigmoid"):
        raise ValueError(f"activation is {activation!r}, expected 'silu' or 'sigmoid'")
    # rows at one stride; or heads of a token side by side, tokens at a stride
    heads = 1
    if x.dim() > 2 and not all(t.is_contiguous() or _row_stride(t) is not None for t in (x, gate)):
        heads = x.shape[-2]
    inner = 2 if heads > 1 else 1
    x, x_ld = _vectors(x, D, heads * D, inner)
    gate, g_ld = _vectors(gate, D, heads * D, inner)
    p = _lib.GatedNormProblem(x.numel() // (heads * D) if heads * D else 0, x_ld, g_ld, heads, D, xd, wd, _ACT[activation], eps)
    return p, x, gate, _on16(weight)


def gated_rms_norm_fwd(x, gate, weight, eps=1e-6, activation="silu", out=None):
    """y = x / sqrt(mean(x^2) + eps) * weight * act(gate) over the last dimension: a mixer's output norm and its gate.

    x, gate [..., D] bf16 or fp16 (typically [B,T,H,D], a norm a head; slices of a projection are read in place); weight
    [D] of x's type or fp32; ``activation`` "silu" or "sigmoid".  ``out`` must not overlap x or gate.
    """
    p, x, gate, weight = _gated_problem(x, gate, weight, eps, activation)
    if out is not None:
        _need(out, "out", x.shape, x.dtype, x)
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _lib.check(_lib.load().gdr_gated_norm_fwd(byref(p), _p(x), _p(gate), _p(weight), _p(y), _s(x)), "gdr_gated_norm_fwd")
    return y


def gated_rms_norm_bwd(x, gate, weight, dy, eps=1e-6, activation="silu"):
    """(dx, dgate, dweight); dweight in weight's type."""
    p, x, gate, weight = _gated_problem(x, gate, weight, eps, activation)
    _need(dy, "dy", x.shape, x.dtype, x, False)
    dy = _on16(dy.contiguous())
    dx, dg = (torch.empty(x.shape, dtype=x.dtype, device=x.device) for _ in range(2))
    dw = torch.empty_like(weight)
    lib = _lib.load()
    ws, n = _workspace(lib.gdr_gated_norm_bwd_workspace_size, p, x)
    _lib.check(lib.gdr_gated_norm_bwd(byref(p), _p(x), _p(gate), _p(weight), _p(dy), _p(dx), _p(dg), _p(dw), _p(ws), n, _s(x)),
               "gdr_gated_norm_bwd")
    return dx, dg, dw


class _GatedRmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, weight, eps, activation):
        ctx.save_for_backward(x, gate, weight)
        ctx.opt = eps, activation
        return gated_rms_norm_fwd(x, gate, weight, eps, activation)

    @staticmethod
    @_once
    def backward(ctx, dy):
        dx, dg, dw = gated_rms_norm_bwd(*ctx.saved_tensors, dy, *ctx.opt)
        return dx, dg, dw, None, None


def gated_rms_norm(x, gate, weight, eps=1e-6, activation="silu"):
    """Differentiable: y.  See gated_rms_norm_fwd."""
    return _GatedRmsNorm.apply(x, gate, weight, eps, activation)


# ---------------------------------------------------------------- norms behind and before a block

def _block_problem(x, h, name, weight, post_weight, gate, gate_activation, residual_scale, eps):
    xd = _tokens(x, "x")
    if x.dim() < 1:
        raise ValueError("x must be [..., D]")
    D = x.shape[-1]
    hd = _dt(h, name, (x.dtype, torch.float32))
    _need(h, name, x.shape, h.dtype, x)
    wd = _dt(weight, "weight", (x.dtype, torch.float32))
    _need(weight, "weight", (D,), weight.dtype, x)
    if post_weight is not None:
        _need(post_weight, "post_weight", (D,), weight.dtype, x)
    if gate_activation not in _ACT:
        raise ValueError(f"gate_activation is {gate_activation!r}, expected None, 'sigmoid' or 'silu'")
    x, x_ld = _vectors(x, D, D, 1)
    g_ld = D
    if gate is not None:
        _need(gate, "gate", x.shape, x.dtype, x, False)
        gate, g_ld = _vectors(gate, D, D, 1)
    elif gate_activation is not None:
        raise ValueError("gate_activation without a gate")
    p = _lib.BlockNormProblem(x.numel() // D if D else 0, x_ld, g_ld, D, xd, wd, hd, _ACT[gate_activation], residual_scale, eps)
    return p, x, _on16(h), gate, _on16(weight), _on16(post_weight)


def block_norm_fwd(x, residual, weight, post_weight=None, gate=None, gate_activation=None, residual_scale=1.0, eps=1e-6,
                   out=None):
    """(y, residual_out) between a block whose output is x and the next one, which reads y:

        b = x / sqrt(mean(x^2) + eps) * post_weight      (x itself without a post_weight)
        residual_out = residual + residual_scale * b * act(gate)
        y = residual_out / sqrt(mean(residual_out^2) + eps) * weight        (from the sum before it is rounded to its type)

    x [..., D] bf16 or fp16; residual [..., D] of x's type or fp32, as residual_out; weight and post_weight [D] of x's type
    or fp32 (both the same); gate [..., D] of x's type through ``gate_activation`` (None: as it is, "sigmoid", "silu").
    ``out`` (for y) must not overlap the inputs.
    """
    p, x, residual, gate, weight, post_weight = _block_problem(x, residual, "residual", weight, post_weight, gate,
                                                               gate_activation, residual_scale, eps)
    if out is not None:
        _need(out, "out", x.shape, x.dtype, x)
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    h = torch.empty(residual.shape, dtype=residual.dtype, device=x.device)
    _lib.check(_lib.load().gdr_block_norm_fwd(byref(p), _p(x), _p(residual), _p(weight), _p(post_weight), _p(gate), _p(y), _p(h),
                                              _s(x)), "gdr_block_norm_fwd")
    return y, h


def block_norm_bwd(x, h, weight, dy, dresidual=None, post_weight=None, gate=None, gate_activation=None, residual_scale=1.0,
                   eps=1e-6):
    """(dx, dresidual_in, dweight, dpost_weight, dgate) at h, the forward's residual_out; ``dresidual`` (h's type) is the
    gradient that reaches it from later layers.  The gradients of what was not given are None."""
    p, x, h, gate, weight, post_weight = _block_problem(x, h, "h", weight, post_weight, gate, gate_activation,
                                                        residual_scale, eps)
    _need(dy, "dy", x.shape, x.dtype, x, False)
    dy = _on16(dy.contiguous())
    if dresidual is not None:
        _need(dresidual, "dresidual", h.shape, h.dtype, x)
        dresidual = _on16(dresidual)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dres = torch.empty(h.shape, dtype=h.dtype, device=x.device)
    dg = None if gate is None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dw = torch.empty_like(weight)
    dp = None if post_weight is None else torch.empty_like(post_weight)
    lib = _lib.load()
    ws, n = _workspace(lib.gdr_block_norm_bwd_workspace_size, p, x)
    _lib.check(lib.gdr_block_norm_bwd(byref(p), _p(x), _p(h), _p(weight), _p(post_weight), _p(gate), _p(dy), _p(dresidual),
                                      _p(dx), _p(dres), _p(dw), _p(dp), _p(dg), _p(ws), n, _s(x)), "gdr_block_norm_bwd")
    return dx, dres, dw, dp, dg


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, post_weight, gate, gate_activation, residual_scale, eps):
        y, h = block_norm_fwd(x, residual, weight, post_weight, gate, gate_activation, residual_scale, eps)
        ctx.save_for_backward(x, h, weight, post_weight, gate)
        ctx.opt = gate_activation, residual_scale, eps
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @_once
    def backward(ctx, dy, dh):
        x, h, weight, post_weight, gate = ctx.saved_tensors
        if dy is None and dh is None:
            return (None,) * 8
        if dy is None:
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        dx, dr, dw, dp, dg = block_norm_bwd(x, h, weight, dy, None if dh is None else dh.contiguous(), post_weight, gate, *ctx.opt)
        return dx, dr, dw, dp, dg, None, None, None


def block_norm(x, residual, weight, post_weight=None, gate=None, gate_activation=None, residual_scale=1.0, eps=1e-6):
    """Differentiable: (y, residual_out).  See block_norm_fwd."""
    return _BlockNorm.apply(x, residual.contiguous(), weight, post_weight, gate, gate_activation, residual_scale, eps)


# ---------------------------------------------------------------- short causal convolution

def _conv_problem(x, weight, bias, activation, cu):
    xd = _tokens(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    B, T, D = x.shape
    wd = _dt(weight, "weight", (x.dtype, torch.float32))
    if weight.dim() != 2 or weight.shape[0] != D or not 2 <= weight.shape[1] <= 4:
        raise ValueError(f"weight has shape {tuple(weight.shape)}, expected ({D}, W) with W from 2 to 4")
    _need(weight, "weight", weight.shape, weight.dtype, x)
    if bias is not None:
        _need(bias, "bias", (D,), weight.dtype, x)
    if activation not in (None, "silu"):
        raise ValueError(f"activation is {activation!r}, expected None or 'silu'")
    _check_cu(cu, x)
    x, ld = _rows(x)
    p = _lib.ConvProblem(B, T, D, weight.shape[1], ld, xd, wd, _p(cu), 0 if cu is None else cu.numel() - 1,
                         _lib.GDR_CONV_SILU if activation else 0)
    return p, x, (B if cu is None else cu.numel() - 1, weight.shape[1] - 1, D)


def short_conv_fwd(x, weight, bias=None, activation=None, initial_state=None, output_final_state=False,
                   cu_seqlens=None, out=None):
    """(y, final_state): every channel of x [B,T,D] with its own W taps, weight [D,W], through SiLU with
    ``activation="silu"``.

    weight and bias [D] in x's type or fp32, 2 <= W <= 4.  ``initial_state`` [N,W-1,D] (x's type, oldest first) holds
    the inputs before each row's (packed: sequence's) first token, None for zeros; final_state, in the same layout,
    the last W-1 inputs (None unless ``output_final_state``).  ``out`` must not overlap x or ``initial_state``.
    """
    cu = _cu(cu_seqlens)
    p, x, sshape = _conv_problem(x, weight, bias, activation, cu)
    if initial_state is not None:
        _need(initial_state, "initial_state", sshape, x.dtype, x)
    if out is not None:
        _need(out, "out", x.shape, x.dtype, x)
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    fin = torch.empty(sshape, dtype=x.dtype, device=x.device) if output_final_state else None
    _lib.check(_lib.load().gdr_conv_fwd(byref(p), _p(x), _p(weight), _p(bias), _p(initial_state), _p(y), _p(fin), _s(x)),
               "gdr_conv_fwd")
    return y, fin


def short_conv_step(x, state, weight, bias=None, activation=None, out=None):
    """y for one new token (or a few) of every row, x [B,T,D]; the cached inputs ``state`` [B,W-1,D] are updated in
    place.  Equals short_conv_fwd over the same tokens."""
    p, x, sshape = _conv_problem(x, weight, bias, activation, None)
    _need(state, "state", sshape, x.dtype, x)
    if out is not None:
        _need(out, "out", x.shape, x.dtype, x)
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _lib.check(_lib.load().gdr_conv_step(byref(p), _p(x), _p(weight), _p(bias), _p(state), _p(y), _s(x)), "gdr_conv_step")
    return y


def short_conv_bwd(x, weight, dy, bias=None, activation=None, initial_state=None, dfinal_state=None, cu_seqlens=None):
    """(dx, dweight, dbias, dinitial_state); dbias is None without a bias, dinitial_state without an initial state."""
    cu = _cu(cu_seqlens)
    p, x, sshape = _conv_problem(x, weight, bias, activation, cu)
    _need(dy, "dy", x.shape, x.dtype, x)
    if initial_state is not None:
        _need(initial_state, "initial_state", sshape, x.dtype, x)
    if dfinal_state is not None:
        _need(dfinal_state, "dfinal_state", sshape, x.dtype, x)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dw = torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    ds = None if initial_state is None else torch.empty_like(initial_state)
    lib = _lib.load()
    ws, n = _workspace(lib.gdr_conv_bwd_workspace_size, p, x)
    _lib.check(lib.gdr_conv_bwd(byref(p), _p(x), _p(weight), _p(bias), _p(dy), _p(initial_state), _p(dfinal_state),
                                _p(dx), _p(dw), _p(db), _p(ds), _p(ws), n, _s(x)), "gdr_conv_bwd")
    return dx, dw, db, ds


class _ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, activation, initial_state, output_final_state, cu_seqlens):
        y, fin = short_conv_fwd(x, weight, bias, activation, initial_state, output_final_state, cu_seqlens)
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.activation = activation
        ctx.set_materialize_grads(False)
        return y, fin

    @staticmethod
    @_once
    def backward(ctx, dy, dfin):
        x, weight, bias, h0, cu = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy.contiguous()
        dx, dw, db, ds = short_conv_bwd(x, weight, dy, bias, ctx.activation, h0,
                                        None if dfin is None else dfin.contiguous(), cu)
        return dx, dw, db, None, ds, None, None


def short_conv(x, weight, bias=None, activation=None, initial_state=None, output_final_state=False, cu_seqlens=None):
    """Differentiable: (y, final_state or None).  See short_conv_fwd."""
    return _ShortConv.apply(x, weight, bias, activation, initial_state, output_final_state, cu_seqlens)


# ---------------------------------------------------------------- selective state space scan

def _scan_problem(x, dt, A, B, C, D, z, dt_bias, dt_softplus, cu):
    xd = _tokens(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    nb, T, width = x.shape
    for name, t in (("A", A), ("B", B), ("C", C)):
        if not isinstance(t, torch.Tensor):
            _check(t, name)
    _need(dt, "dt", x.shape, x.dtype, x, False)
    if z is not None:
        _need(z, "z", x.shape, x.dtype, x, False)
    if A.dim() != 2 or A.shape[0] != width:
        raise ValueError(f"A has shape {tuple(A.shape)}, expected ({width}, N)")
    N = A.shape[1]
    _need(A, "A", (width, N), torch.float32, x)
    if B.dim() != 4:
        raise ValueError(f"B has shape {tuple(B.shape)}, expected ({nb}, {T}, G, {N})")
    _need(B, "B", (nb, T, B.shape[2], N), x.dtype, x, False)
    _need(C, "C", B.shape, x.dtype, x, False)
    if D is not None:
        _need(D, "D", (width,), torch.float32, x)
    if dt_bias is not None:
        _need(dt_bias, "dt_bias", (width,), torch.float32, x)
    _check_cu(cu, x)
    x, x_ld = _rows(x)
    dt, dt_ld = _rows(dt)
    z, z_ld = (None, width) if z is None else _rows(z)
    B, b_ld = _rows(B, 2)
    C, c_ld = _rows(C, 2)
    p = _lib.ScanProblem(nb, T, width, N, B.shape[2], x_ld, dt_ld, z_ld, b_ld, c_ld, xd, _p(cu),
                         0 if cu is None else cu.numel() - 1, _lib.GDR_SCAN_DT_SOFTPLUS if dt_softplus else 0)
    return p, x, dt, B, C, z, (nb if cu is None else cu.numel() - 1, width, N)


def selective_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False, initial_state=None,
                       output_final_state=True, cu_seqlens=None, save_for_backward=False, out=None):
    """(y, final_state, saved) of the diagonal state space model of every channel d of x [B,T,D]:

        delta_t = dt_t + dt_bias (through softplus with ``dt_softplus``)
        h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t        (N states a channel, fp32)
        y_t = (C_t . h_t + D x_t) * silu(z_t)                  (D and z optional)

    x, dt, z [B,T,D] and B, C [B,T,G,N] (channel d reads group d // (D/G)) in bf16 or fp16; A [D,N], D [D], dt_bias [D]
    and the states [N_seqs,D,N] fp32; 1 <= N <= 64.  ``saved`` (the states before every few tokens; None unless
    ``save_for_backward``) is what selective_scan_bwd needs.
    """
    cu = _cu(cu_seqlens)
    p, x, dt, B, C, z, sshape = _scan_problem(x, dt, A, B, C, D, z, dt_bias, dt_softplus, cu)
    if initial_state is not None:
        _need(initial_state, "initial_state", sshape, torch.float32, x)
    if out is not None:
        _need(out, "out", x.shape, x.dtype, x)
    lib = _lib.load()
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    fin = torch.empty(sshape, dtype=torch.float32, device=x.device) if output_final_state else None
    saved = _workspace(lib.gdr_scan_saved_bytes, p, x)[0] if save_for_backward else None
    n = c_size_t(0)
    _lib.check(lib.gdr_scan_workspace_size(byref(p), 0, byref(n)), "gdr_scan_workspace_size")
    ws = torch.empty(n.value, dtype=torch.uint8, device=x.device) if n.value else None
    _lib.check(lib.gdr_scan_fwd(byref(p), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(z), _p(dt_bias),
                                _p(initial_state), _p(y), _p(fin), _p(saved), _p(ws), n.value, _s(x)), "gdr_scan_fwd")
    return y, fin, saved


def selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus=False, out=None):
    """y for one new token (or a few) of every row; ``state`` [B,D,N] fp32 is updated in place.  Equals
    selective_scan_fwd over the same tokens."""
    p, x, dt, B, C, z, sshape = _scan_problem(x, dt, A, B, C, D, z, dt_bias, dt_softplus, None)
    _need(state, "state", sshape, torch.float32, x)
    if out is not None:
        _need(out, "out", x.shape, x.dtype, x)
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _lib.check(_lib.load().gdr_scan_step(byref(p), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(z), _p(dt_bias),
                                         _p(state), _p(y), _s(x)), "gdr_scan_step")
    return y


def selective_scan_bwd(x, dt, A, B, C, dy, saved, D=None, z=None, dt_bias=None, dt_softplus=False, initial_state=None,
                       dfinal_state=None, cu_seqlens=None):
    """(dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dinitial_state); the gradients of arguments that were not given are None.

    ``saved`` is what selective_scan_fwd returned for the same inputs.  dx, ddt, dz, dB, dC have the tokens' type, the
    others fp32."""
    cu = _cu(cu_seqlens)
    p, x, dt, B, C, z, sshape = _scan_problem(x, dt, A, B, C, D, z, dt_bias, dt_softplus, cu)
    _need(dy, "dy", x.shape, x.dtype, x)
    if initial_state is not None:
        _need(initial_state, "initial_state", sshape, torch.float32, x)
    if dfinal_state is not None:
        _need(dfinal_state, "dfinal_state", sshape, torch.float32, x)
    _check(saved, "saved", None, torch.uint8, x)
    lib = _lib.load()
    n = c_size_t(0)
    _lib.check(lib.gdr_scan_saved_bytes(byref(p), byref(n)), "gdr_scan_saved_bytes")
    if saved.numel() < n.value:
        raise ValueError(f"saved holds {saved.numel()} bytes, this problem needs {n.value}")

    def like(t):
        return None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device)

    dx, ddt, dA, dB, dC, dD, dz, dbias, ds = (like(t) for t in (x, dt, A, B, C, D, z, dt_bias, initial_state))
    _lib.check(lib.gdr_scan_workspace_size(byref(p), 1, byref(n)), "gdr_scan_workspace_size")
    ws = torch.empty(n.value, dtype=torch.uint8, device=x.device)
    _lib.check(lib.gdr_scan_bwd(byref(p), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(z), _p(dt_bias), _p(dy),
                                _p(initial_state), _p(dfinal_state), _p(saved), _p(dx), _p(ddt), _p(dA), _p(dB), _p(dC),
                                _p(dD), _p(dz), _p(dbias), _p(ds), _p(ws), n.value, _s(x)), "gdr_scan_bwd")
    return dx, ddt, dA, dB, dC, dD, dz, dbias, ds


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, output_final_state, cu_seqlens):
        y, fin, saved = selective_scan_fwd(x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state,
                                           output_final_state, cu_seqlens, save_for_backward=True)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens, saved)
        ctx.softplus = dt_softplus
        ctx.set_materialize_grads(False)
        return y, fin

    @staticmethod
    @_once
    def backward(ctx, dy, dfin):
        x, dt, A, B, C, D, z, dt_bias, h0, cu, saved = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy.contiguous()
        dx, ddt, dA, dB, dC, dD, dz, dbias, ds = selective_scan_bwd(
            x, dt, A, B, C, dy, saved, D, z, dt_bias, ctx.softplus, h0, None if dfin is None else dfin.contiguous(), cu)
        return dx, ddt, dA, dB, dC, dD, dz, dbias, None, ds, None, None


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False, initial_state=None,
                   output_final_state=False, cu_seqlens=None):
    """Differentiable: (y, final_state or None).  See selective_scan_fwd."""
    return _SelectiveScan.apply(x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, output_final_state,
                                cu_seqlens)
