"""Linear attention with one decay a head: the delta rule's sibling without its correction.

Python surface of ``gdr_lin_*`` in ``include/gdr.h``: ``linear_attention_fwd`` / ``_bwd`` / ``_step`` map onto one library
call each and ``linear_attention`` is differentiable (once).  Token tensors may be row-strided views (slices of a fused
projection are read in place where their rows lie on 16-byte boundaries); any other view is copied.
"""

from __future__ import annotations

from ctypes import byref, c_size_t

import torch

from . import _lib
from ._args import _check, _check_cu, _cu, _need, _rows
from .layer_ops import _on16, _once, _p, _s, _tokens

__all__ = ["linear_attention", "linear_attention_fwd", "linear_attention_bwd", "linear_attention_step"]


def _aligned(t, ld):
    """(t, ld) with rows on 16-byte boundaries."""
    if ld % 8 or t.data_ptr() % 16:
        t = t.clone(memory_format=torch.contiguous_format)  # (contiguous() hands a misaligned one back)
        ld = t.shape[-1] * t.shape[-2]
    return t, ld


def _problem(q, k, v, decay, scale, cu, step=False):
    qd = _tokens(q, "q")
    if q.dim() != 4 or not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("q, k and v must be [B, T, H, D]")
    B, T, Hk, K = q.shape
    H, V = v.shape[2], v.shape[3]
    _need(k, "k", q.shape, q.dtype, q, False)
    _need(v, "v", (B, T, H, V), q.dtype, q, False)
    _need(decay, "decay", (H,), torch.float32, q)
    if decay.requires_grad and torch.is_grad_enabled():
        raise ValueError("decay is a constant of the heads: it has no gradient (detach it)")
    _check_cu(cu, q)
    (q, q_ld), (k, k_ld), (v, v_ld) = _rows(q, 2), _rows(k, 2), _rows(v, 2)
    if not step:
        (q, q_ld), (k, k_ld), (v, v_ld) = _aligned(q, q_ld), _aligned(k, k_ld), _aligned(v, v_ld)
    n = 0 if cu is None else cu.numel() - 1
    p = _lib.LinProblem(B, T, Hk, H, K, V, q_ld, k_ld, v_ld, qd, K ** -0.5 if scale is None else scale, _p(cu), n)
    return p, q, k, v, (B if cu is None else n, H, K, V)


def _lin_workspace(lib, p, backward, like):
    n = c_size_t(0)
    _lib.check(lib.gdr_lin_workspace_size(byref(p), backward, byref(n)), "gdr_lin_workspace_size")
    return (torch.empty(n.value, dtype=torch.uint8, device=like.device) if n.value else None), n.value


def linear_attention_fwd(q, k, v, decay, scale=None, initial_state=None, output_final_state=False, cu_seqlens=None,
                         out=None):
    """(o, final_state) of every head's  S_t = exp(decay) S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t.

    q, k [B,T,Hk,K] and v [B,T,H,V] bf16 or fp16 (head j reads q/k head j // (H/Hk)), K and V from 8 to 128 in steps of 8;
    ``decay`` [H] fp32, at most 0: a constant of the heads, without a gradient; ``scale`` is K ** -0.5 unless given.
    ``initial_state`` [N,H,K,V] fp32 (None: zeros) and final_state (None unless ``output_final_state``): one a row, or a
    sequence of a packed batch (``cu_seqlens``).  ``out`` must not overlap q, k or v.  States may be of any size; with fp16
    the products scale q.k (backwards also scale do.v) have to stay within 65504.
    """
    cu = _cu(cu_seqlens)
    p, q, k, v, sshape = _problem(q, k, v, decay, scale, cu)
    if initial_state is not None:
        _need(initial_state, "initial_state", sshape, torch.float32, q)
        initial_state = _on16(initial_state)
    if out is not None:
        _need(out, "out", v.shape, v.dtype, q)
    lib = _lib.load()
    o = out if out is not None else torch.empty(v.shape, dtype=v.dtype, device=v.device)
    fin = torch.empty(sshape, dtype=torch.float32, device=q.device) if output_final_state else None
    ws, n = _lin_workspace(lib, p, 0, q)
    _lib.check(lib.gdr_lin_fwd(byref(p), _p(q), _p(k), _p(v), _p(decay), _p(initial_state), _p(o), _p(fin), _p(ws), n,
                               _s(q)), "gdr_lin_fwd")
    return o, fin


def linear_attention_step(q, k, v, decay, state, scale=None, out=None):
    """o for one new token (or a few) of every row; ``state`` [B,H,K,V] fp32 is updated in place.  Equals
    linear_attention_fwd over the same tokens up to rounding (fp32 throughout: no product of 16-bit numbers)."""
    p, q, k, v, sshape = _problem(q, k, v, decay, scale, None, step=True)
    _need(state, "state", sshape, torch.float32, q)
    if out is not None:
        _need(out, "out", v.shape, v.dtype, q)
    o = out if out is not None else torch.empty(v.shape, dtype=v.dtype, device=v.device)
    _lib.check(_lib.load().gdr_lin_step(byref(p), _p(q), _p(k), _p(v), _p(decay), _p(state), _p(o), _s(q)), "gdr_lin_step")
    return o


def linear_attention_bwd(q, k, v, decay, do, scale=None, initial_state=None, dfinal_state=None, cu_seqlens=None):
    """(dq, dk, dv, dinitial_state); dinitial_state is None without an initial state.  ``do`` [B,T,H,V] in v's type,
    ``dfinal_state`` fp32 as the states (None: zeros)."""
    cu = _cu(cu_seqlens)
    p, q, k, v, sshape = _problem(q, k, v, decay, scale, cu)
    _need(do, "do", v.shape, v.dtype, q)
    do, _ = _aligned(do, v.shape[2] * v.shape[3])
    for name, t in (("initial_state", initial_state), ("dfinal_state", dfinal_state)):
        if t is not None:
            _need(t, name, sshape, torch.float32, q)
    initial_state, dfinal_state = _on16(initial_state), _on16(dfinal_state)
    lib = _lib.load()
    dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
    ds = None if initial_state is None else torch.empty_like(initial_state)
    ws, n = _lin_workspace(lib, p, 1, q)
    _lib.check(lib.gdr_lin_bwd(byref(p), _p(q), _p(k), _p(v), _p(decay), _p(do), _p(initial_state), _p(dfinal_state), _p(dq),
                               _p(dk), _p(dv), _p(ds), _p(ws), n, _s(q)), "gdr_lin_bwd")
    return dq, dk, dv, ds


class _LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, decay, scale, initial_state, output_final_state, cu_seqlens):
        o, fin = linear_attention_fwd(q, k, v, decay, scale, initial_state, output_final_state, cu_seqlens)
        ctx.save_for_backward(q, k, v, decay, initial_state, cu_seqlens)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return o, fin

    @staticmethod
    @_once
    def backward(ctx, do, dfin):
        q, k, v, decay, h0, cu = ctx.saved_tensors
        do = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if do is None else do.contiguous()
        dq, dk, dv, ds = linear_attention_bwd(q, k, v, decay, do, ctx.scale, h0, None if dfin is None else dfin.contiguous(), cu)
        return dq, dk, dv, None, None, ds, None, None


def linear_attention(q, k, v, decay, scale=None, initial_state=None, output_final_state=False, cu_seqlens=None):
    """Differentiable: (o, final_state or None).  See linear_attention_fwd."""
    if isinstance(decay, torch.Tensor) and decay.requires_grad and torch.is_grad_enabled():
        raise ValueError("decay is a constant of the heads: it has no gradient (detach it)")
    return _LinearAttention.apply(q, k, v, decay, scale, initial_state, output_final_state, cu_seqlens)
