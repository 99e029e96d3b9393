"""Layer norm of token rows, and its gradient.

Tensor checks and descriptors for ``cp_layer_norm_fwd`` / ``cp_layer_norm_bwd``
(``include/cpattn.h``); :func:`vlm_zigzag_head_gb300.autograd.layer_norm` is the
differentiable form.
"""
from __future__ import annotations

import functools
from typing import Optional

import torch

from . import CP_F32, CpError, _binding as _b, _dt
from .norm_rope import _at, _on_device, _raw_stream


def _rows(x: torch.Tensor, name: str) -> torch.Tensor:
    """x as ``[T, D]`` with contiguous rows (a copy only where no view does)."""
    if x.dim() < 1:
        raise CpError(2, "%s must have at least one dimension" % name)
    if not x.is_cuda:
        raise CpError(1, "tensors must live on a CUDA device")
    if x.dim() != 2:
        x = x.reshape(-1, x.shape[-1]) if x.numel() else x.new_empty((0, x.shape[-1]))
    if x.shape[1] > 1 and x.stride(1) != 1:
        x = x.contiguous()
    return x


@functools.lru_cache(maxsize=256)
def _desc(dtype, w_dtype, T, D, x_stride, dy_stride, eps):
    f = _b.LayerNormDesc()
    if T > 0x7fffffff:
        raise CpError(2, "at most 2^31 - 1 rows")
    f.dtype, f.weight_dtype = dtype, w_dtype
    f.T, f.D = T, D
    # the stride of a dimension of one element is never used
    f.x_stride, f.dy_stride = (x_stride, dy_stride) if T > 1 else (D, D)
    f.eps = eps
    f.workspace = {}   # the backward's bytes by device, as they get known
    return f


def _prepare(x, weight, bias, eps, dy=None):
    """The checked descriptor of rows ``x [T, D]``."""
    w_dtype, (T, D), device = CP_F32, x.shape, x.device
    for w in (weight, bias):
        if w is None:
            continue
        if w.shape != (D,) or w.device != device or not w.is_contiguous():
            raise CpError(2, "weight and bias must be contiguous [D] tensors on x's device")
        w_dtype = _dt(w)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise CpError(3, "weight and bias must share a dtype")
    dy_stride = 0
    if dy is not None:
        if dy.shape != x.shape or dy.dtype != x.dtype or dy.device != device:
            raise CpError(2, "dy must match x")
        dy_stride = dy.stride(0)
    return _desc(_dt(x), w_dtype, T, D, x.stride(0), dy_stride, float(eps))


def cp_layer_norm_fwd(x, weight=None, bias=None, eps: float = 1e-5):
    """Layer norm of the last dimension of ``x [..., D]`` (bf16 or fp32; rows of any
    stride, D up to 16384); ``weight`` / ``bias``: ``[D]`` (bf16 or fp32) or None.
    Returns ``(y, mean, rstd)``: y contiguous; mean and rstd fp32, one per row, for
    :func:`cp_layer_norm_bwd`."""
    rows = _rows(x, "x")
    return _launch_fwd(_prepare(rows, weight, bias, eps), rows, weight, bias, x.shape)


def _launch_fwd(f, rows, weight, bias, shape, stats=True):
    device = rows.device
    y = torch.empty(shape, dtype=rows.dtype, device=device)
    mean = rstd = None
    if stats:
        mean = torch.empty(shape[:-1], dtype=torch.float32, device=device)
        rstd = torch.empty_like(mean)
    with _on_device(device):
        _b.check(_b.lib().cp_layer_norm_fwd(
            f, rows.data_ptr(), _at(weight), _at(bias), y.data_ptr(), _at(mean), _at(rstd),
            _raw_stream(device)))
    return y, mean, rstd


def cp_layer_norm_bwd(x, dy, mean, rstd, weight=None, *, bias_grad: bool = False,
                      weight_grad: Optional[bool] = None, input_grad: bool = True):
    """Gradient of :func:`cp_layer_norm_fwd`: ``(dx, dweight, dbias)``, each None where
    not wanted (``weight_grad`` defaults to whether there is a weight).  ``dy``: any strides,
    x's dtype.  dx is contiguous in x's dtype, dweight and dbias are fp32 ``[D]``."""
    rows, g = _rows(x, "x"), _rows(dy, "dy")
    f = _prepare(rows, weight, None, 0.0, g)
    T, device = f.T, x.device
    for s in (mean, rstd):
        if s.numel() != T or s.dtype != torch.float32 or s.device != device or \
                not s.is_contiguous():
            raise CpError(2, "mean and rstd must be those of the forward")
    if weight_grad is None:
        weight_grad = weight is not None
    return _launch_bwd(f, rows, g, mean, rstd, weight, input_grad, weight_grad, bias_grad, x.shape)


def _launch_bwd(f, rows, dy, mean, rstd, weight, input_grad, weight_grad, bias_grad, shape):
    device = rows.device
    dx = torch.empty(shape, dtype=rows.dtype, device=device) if input_grad else None
    dw = torch.empty(f.D, dtype=torch.float32, device=device) if weight_grad else None
    db = torch.empty(f.D, dtype=torch.float32, device=device) if bias_grad else None
    lib = _b.lib()
    with _on_device(device):
        ws, nbytes = None, 0
        if weight_grad or bias_grad:
            nbytes = f.workspace.get(device.index)
            if nbytes is None:
                nbytes = f.workspace[device.index] = lib.cp_layer_norm_bwd_workspace_size(f)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _b.check(lib.cp_layer_norm_bwd(
            f, rows.data_ptr(), dy.data_ptr(), _at(weight), mean.data_ptr(), rstd.data_ptr(),
            _at(dx), _at(dw), _at(db), _at(ws), nbytes, _raw_stream(device)))
    return dx, dw, db
