"""Argument checks and marshalling that the package's operators share."""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib

_DT = {torch.bfloat16: _lib.GDR_BF16, torch.float16: _lib.GDR_FP16, torch.float32: _lib.GDR_FP32}


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(t, name, shape=None, dtype=None, like=None, optional=False, contiguous=True):
    """The library reads and writes every tensor through a raw device pointer as a contiguous row-major array
    of the problem's shape: anything else is refused here, before a kernel could read past its end."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if like is not None and t.get_device() != like.get_device():
        raise ValueError(f"{name} is on {t.device}, the other tensors on {like.device}")
    if shape is not None and t.shape != shape:  # (a torch.Size is a tuple)
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need(t, name, shape, dtype, like, contiguous=True):
    """_check of a required tensor with everything given: one quick test, and _check for the message when it fails."""
    try:
        ok = t.shape == shape and t.dtype == dtype and t.get_device() == like.get_device() and (
            not contiguous or t.is_contiguous())
    except AttributeError:
        ok = False
    if not ok:
        _check(t, name, shape, dtype, like, contiguous=contiguous)


def _check_cu(cu, q):
    if cu is not None:
        _check(cu, "cu_seqlens", (cu.numel(),), torch.int32, q)
        if q.shape[0] != 1:
            raise ValueError("a packed batch (cu_seqlens) has B = 1")


def _cu(cu_seqlens):
    if cu_seqlens is None:
        return None
    if cu_seqlens.dtype != torch.int32:
        cu_seqlens = cu_seqlens.to(torch.int32)
    return cu_seqlens.contiguous()


def _row_stride(t, inner=1):
    """The one stride at which a tensor's rows (its last ``inner`` dimensions, contiguous) follow one another, or None."""
    n = 1
    for d in t.shape[t.dim() - inner:]:
        n *= d
    lead = t.dim() - inner
    want, ok = 1, True
    for i in range(t.dim() - 1, lead - 1, -1):
        ok = ok and (t.shape[i] == 1 or t.stride(i) == want)
        want *= t.shape[i]
    ld = None
    for i in range(lead - 1, -1, -1):
        if t.shape[i] == 1:
            continue
        if ld is None:
            ld = step = t.stride(i)
        ok = ok and t.stride(i) == step
        step = t.stride(i) * t.shape[i]
    ld = n if ld is None else ld
    return ld if ok and ld >= n else None


def _rows(t, inner=1):
    """(t, row stride): a tensor whose last ``inner`` dimensions are contiguous and whose rows follow one another at
    one stride (a slice of a fused projection is one); any other view is copied."""
    if not t.is_contiguous():
        ld = _row_stride(t, inner)
        if ld is not None:
            return t, ld
        t = t.contiguous()
    return t, t.shape[-1] if inner == 1 else t.shape[-1] * t.shape[-2]
