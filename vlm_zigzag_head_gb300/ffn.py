"""Gated feed-forward block, and its gradient.

Tensor checks and descriptors for ``cp_gated_ffn_fwd`` / ``cp_gated_ffn_bwd``
(``include/cpattn.h``); :func:`vlm_zigzag_head_gb300.autograd.gated_ffn` is the
differentiable form.
"""
from __future__ import annotations

import functools
from typing import Optional, Sequence

import torch

from . import CP_BF16, CP_F32, CpError, Workspace, _binding as _b, _dt
from .layer_norm import _rows
from .norm_rope import _at, _on_device, _raw_stream
from .scored import _like, _space

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
_GRAD_DTYPES = {torch.bfloat16: CP_BF16, torch.float32: CP_F32}


def _aligned(x: torch.Tensor) -> torch.Tensor:
    """x, or a copy whose rows are contiguous, apart, and lie on 16-byte boundaries."""
    per16 = 16 // x.element_size()
    if x.dim() >= 1 and x.stride(-1) == 1 and x.data_ptr() % 16 == 0 and \
            all(s % per16 == 0 and s >= x.shape[-1] for s, n in zip(x.stride()[:-1], x.shape)
                if n > 1):
        return x
    x = x.contiguous()
    return x if x.data_ptr() % 16 == 0 else x.clone()


@functools.lru_cache(maxsize=256)
def _desc(dtype, grad_dtype, activation, T, D, F, D_out, x_stride, wg_stride, wu_stride,
          wd_stride, dy_stride):
    """The descriptor, and its workspace and kept sizes as they get known."""
    if T > 0x7fffffff:
        raise CpError(2, "at most 2^31 - 1 rows")
    f = _b.GatedFfnDesc()
    f.dtype, f.grad_dtype, f.activation = dtype, grad_dtype, activation
    f.T, f.D, f.F, f.D_out = T, D, F, D_out
    f.x_stride, f.dy_stride = (x_stride, dy_stride) if T > 1 else (D, D_out)
    f.w_gate_stride, f.w_up_stride, f.w_down_stride = wg_stride, wu_stride, wd_stride
    return f, {}


def _kept_bytes(f, sizes):
    if "kept" not in sizes:
        sizes["kept"] = _b.lib().cp_gated_ffn_kept_size(f)
    return sizes["kept"]


def _workspace_bytes(f, sizes, device, backward):
    key = device.index, backward
    if key not in sizes:
        L = _b.lib()
        size = L.cp_gated_ffn_bwd_workspace_size if backward else \
            L.cp_gated_ffn_fwd_workspace_size
        got = size(f)
        if got == 0:
            raise CpError(2, L.cp_last_error().decode(errors="replace"))
        sizes[key] = got
    return sizes[key]


def _prepare(x, w_gate, w_up, w_down, activation, grad_dtype, dy=None):
    """The checked descriptor of rows ``x [T, D]``, with its workspace sizes."""
    code, hidden, out = ACTIVATIONS.get(activation), w_gate.shape, w_down.shape
    if code is None:
        raise CpError(1, "activation must be one of %s" % ", ".join(ACTIVATIONS))
    if len(hidden) != 2 or len(out) != 2 or hidden != w_up.shape or hidden[1] != x.shape[1] or \
            out[1] != hidden[0]:
        raise CpError(2, "w_gate and w_up must be [F, D], w_down [D_out, F]")
    (T, D), F, D_out, dtype, device = x.shape, hidden[0], out[0], x.dtype, x.device
    strides = []
    for w, width in ((w_gate, D), (w_up, D), (w_down, F)):
        if w.dtype != dtype:
            raise CpError(3, "x and the weights must share a dtype")
        if w.device != device:
            raise CpError(1, "x and the weights must share a device")
        row, column = w.stride()
        if width > 1 and column != 1:
            raise CpError(1, "the last dimension of the weights must be contiguous")
        strides.append(row)
    if dy is not None and (dy.shape != (T, D_out) or dy.dtype != dtype or dy.device != device):
        raise CpError(2, "dy must match y")
    return _desc(_dt(x), grad_dtype, code, T, D, F, D_out, x.stride(0), *strides,
                 D_out if dy is None else dy.stride(0))


def cp_gated_ffn_fwd(x, w_gate, w_up, w_down, activation: str = "silu", *, keep: bool = False,
                     workspace: Optional[Workspace] = None):
    """``y = (a(x w_gate^T) * (x w_up^T)) w_down^T`` of the last dimension of ``x [..., D]``
    (fp32 stays fp32: beyond 64 rows on the tensor cores too, as sums of bf16 parts that lose
    no digit), with ``w_gate``/``w_up [F, D]``, ``w_down [D_out, F]`` and ``a`` one of
    ``"silu"``, ``"gelu"``, ``"gelu_tanh"``.  D, F, D_out: multiples of
    8; rows of any stride that lie on 16-byte boundaries.  With ``keep`` returns ``(y, gate,
    up)``, the two projections for :func:`cp_gated_ffn_bwd` as byte tensors in the library's
    layout (bf16: to 24 bits).  Without ``workspace`` each call takes one of its own, so calls
    on several streams may overlap; whether a bounded device wait ran out, which leaves results
    unwritten, is known from a caller's workspace alone (:func:`cp_workspace_status`)."""
    rows = _rows(x, "x")
    f, sizes = _prepare(rows, w_gate, w_up, w_down, activation, _dt(rows))
    device, lead = x.device, x.shape[:-1]
    y = torch.empty((*lead, f.D_out), dtype=x.dtype, device=device)
    gate = up = None
    if keep:
        gate, up = (torch.empty(_kept_bytes(f, sizes), dtype=torch.uint8, device=device)
                    for _ in range(2))
    with _on_device(device):
        ws, ptr, size = _space(workspace, _workspace_bytes(f, sizes, device, False), device)
        _b.check(_b.lib().cp_gated_ffn_fwd(
            f, rows.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
            y.data_ptr(), _at(gate), _at(up), ptr, size, _raw_stream(device)))
    return (y, gate, up) if keep else y


def cp_gated_ffn_bwd(x, w_gate, w_up, w_down, gate, up, dy, activation: str = "silu", *,
                     grad_dtype=torch.float32, wanted: Sequence[bool] = (True,) * 4,
                     workspace: Optional[Workspace] = None):
    """Gradient of :func:`cp_gated_ffn_fwd` (``gate``, ``up``: what it kept): ``(dx, dw_gate,
    dw_up, dw_down)``, None where ``wanted`` says so.  dx has x's dtype; the weights'
    gradients have ``grad_dtype``: fp32, or bf16 for bf16 inputs.  ``workspace`` as in the forward."""
    if len(wanted) != 4:
        raise CpError(2, "wanted must say yes or no to dx, dw_gate, dw_up and dw_down")
    rows, g = _rows(x, "x"), _rows(dy, "dy")
    if grad_dtype not in _GRAD_DTYPES:
        raise CpError(3, "dtype %s not supported (bf16 or fp32)" % grad_dtype)
    f, sizes = _prepare(rows, w_gate, w_up, w_down, activation, _GRAD_DTYPES[grad_dtype], g)
    device = x.device
    for t, name in ((gate, "gate"), (up, "up")):
        _like(t, (_kept_bytes(f, sizes),), torch.uint8, device, name)
        if not t.is_contiguous():
            raise CpError(1, "%s must be contiguous" % name)
    like = ((x, x.dtype), (w_gate, grad_dtype), (w_up, grad_dtype), (w_down, grad_dtype))
    out = [torch.empty(t.shape, dtype=dt, device=device) if on else None
           for (t, dt), on in zip(like, wanted)]
    with _on_device(device):
        ws, ptr, size = _space(workspace, _workspace_bytes(f, sizes, device, True), device)
        _b.check(_b.lib().cp_gated_ffn_bwd(
            f, rows.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
            gate.data_ptr(), up.data_ptr(), g.data_ptr(), *(_at(t) for t in out), ptr, size,
            _raw_stream(device)))
    return tuple(out)
