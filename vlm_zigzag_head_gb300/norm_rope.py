"""RMS norm of query and key heads with the position rotation, and its gradient.

Tensor checks and descriptors for ``cp_qk_norm_rope_fwd`` / ``cp_qk_norm_rope_bwd``
(``include/cpattn.h``); :func:`vlm_zigzag_head_gb300.autograd.qk_norm_rope` is the
differentiable form.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence

import torch
from torch.autograd import forward_ad

from . import CP_F32, CpError, _binding as _b, _dt


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _raw_stream(device) -> int:
    """The current stream's handle (without building a Stream object per call)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _wants_grad(*tensors) -> bool:
    """Whether autograd has to know of the call: for a backward to follow, or, with a dual
    tensor, for the autograd function to say that it has no forward-mode rule (a plain call
    would drop the tangent, which reads as a derivative of zero)."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        return True
    # no dual tensor outside a level; the private number saves a query per tensor
    return getattr(forward_ad, "_current_level", 0) >= 0 and any(
        t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


class _on_device:
    """``torch.cuda.device``, free of charge where the device is current already."""

    def __init__(self, device):
        other = torch._C._cuda_getDevice() != device.index
        self._guard = torch.cuda.device(device) if other else None

    def __enter__(self):
        if self._guard is not None:
            self._guard.__enter__()

    def __exit__(self, *exc):
        if self._guard is not None:
            self._guard.__exit__(*exc)


def _check_heads(x, name, like=None):
    if x.dim() != 3:
        raise CpError(2, "%s must be [T, heads, d]" % name)
    if not x.is_cuda:
        raise CpError(1, "tensors must live on a CUDA device")
    if like is not None and (x.device != like.device or x.dtype != like.dtype):
        raise CpError(2, "q and k must share device and dtype")


@functools.lru_cache(maxsize=256)
def _desc(dtype, q_shape, q_stride, k_shape, k_stride, pos_shape, w_dtype, eps, theta, rot_dim,
          sections, interleaved, inv_freq):
    """The checked descriptor of one set of shapes and options."""
    T, H, d = q_shape
    if k_shape[0] != T or k_shape[2] != d:
        raise CpError(2, "q and k must share tokens and head size")
    if d > 1 and (q_stride[2] != 1 or k_stride[2] != 1):
        raise CpError(1, "the last dimension of q and k must be contiguous")
    rot = d if rot_dim is None else int(rot_dim)
    if rot < 0 or rot > d or rot % 16:
        raise CpError(2, "rot_dim must be a multiple of 16 in [0, head_dim]")
    axes = pos_shape[0] if len(pos_shape) == 2 else 1
    if len(pos_shape) not in (1, 2) or pos_shape[-1] != T or not 1 <= axes <= 4:
        raise CpError(2, "positions must be [T] or [axes, T] with at most 4 axes")
    if sections is None:
        if axes != 1:
            raise CpError(2, "several position axes need sections")
        sections = (rot // 2,)
    if len(sections) != axes:
        raise CpError(2, "sections must have one entry per position axis")
    if inv_freq is None:
        if not theta > 0:
            raise CpError(1, "theta must be positive")
        inv_freq = [theta ** (-2.0 * p / rot) for p in range(rot // 2)]
    elif len(inv_freq) != rot // 2:
        raise CpError(2, "inv_freq must have rot_dim / 2 entries")
    f = _b.NormRopeDesc()
    f.dtype, f.weight_dtype = dtype, w_dtype
    f.T, f.H, f.H_kv, f.d = T, H, k_shape[1], d
    # the stride of a dimension of one element is never used
    f.q_stride_t, f.q_stride_h = (s if n > 1 else 0 for s, n in zip(q_stride, q_shape[:2]))
    f.k_stride_t, f.k_stride_h = (s if n > 1 else 0 for s, n in zip(k_stride, k_shape[:2]))
    f.rot_dim, f.interleaved, f.n_axes = rot, int(interleaved), axes
    for i, n in enumerate(sections):
        f.sections[i] = n
    f.inv_freq = (ctypes.c_double * max(1, len(inv_freq)))(*inv_freq)
    f.eps = eps
    return f


def _prepare(q, k, positions, q_weight, k_weight, eps, theta, rot_dim, sections, interleaved,
             inv_freq):
    _check_heads(q, "q")
    _check_heads(k, "k", q)
    if positions.dtype != torch.int32 or positions.device != q.device or \
            not positions.is_contiguous():
        raise CpError(3, "positions must be a contiguous int32 tensor on q's device")
    w_dtype = CP_F32
    for w in (q_weight, k_weight):
        if w is None:
            continue
        if w.shape != q.shape[2:] or w.device != q.device or not w.is_contiguous():
            raise CpError(2, "norm weights must be contiguous [head_dim] tensors on q's device")
        w_dtype = _dt(w)
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise CpError(3, "the norm weights must share a dtype")
    return _desc(_dt(q), tuple(q.shape), q.stride(), tuple(k.shape), k.stride(),
                 tuple(positions.shape), w_dtype, float(eps), float(theta), rot_dim,
                 None if sections is None else tuple(int(n) for n in sections), bool(interleaved),
                 None if inv_freq is None else tuple(float(x) for x in inv_freq))


def cp_qk_norm_rope_fwd(q, k, positions, q_weight=None, k_weight=None, eps: float = 1e-6,
                        theta: float = 10000.0, rot_dim: Optional[int] = None,
                        sections: Optional[Sequence[int]] = None, interleaved: bool = False,
                        inv_freq: Optional[Sequence[float]] = None):
    """Norm and rotate every head of ``q [T,H,d]`` and ``k [T,H_kv,d]`` (bf16 or
    fp32; any token and head strides, e.g. slices of one projection's output).

    ``positions``: int32 ``[T]``, or ``[axes, T]`` with ``sections`` giving the
    number of rotated pairs that read each axis.  ``rot_dim`` (default: the
    whole head): rotated elements of each head; pair p turns by its position
    times ``inv_freq[p]`` (default ``theta ** (-2 p / rot_dim)``).
    ``q_weight`` / ``k_weight``: norm weights ``[d]`` (bf16 or fp32) or None.
    Returns contiguous ``(q_out, k_out)``."""
    f = _prepare(q, k, positions, q_weight, k_weight, eps, theta, rot_dim, sections,
                 interleaved, inv_freq)
    return _launch_fwd(f, q, k, positions, q_weight, k_weight)


def _launch_fwd(f, q, k, positions, q_weight, k_weight):
    device = q.device
    q_out = torch.empty(q.shape, dtype=q.dtype, device=device)
    k_out = torch.empty(k.shape, dtype=k.dtype, device=device)
    with _on_device(device):
        _b.check(_b.lib().cp_qk_norm_rope_fwd(
            f, q.data_ptr(), k.data_ptr(), positions.data_ptr(), _at(q_weight), _at(k_weight),
            q_out.data_ptr(), k_out.data_ptr(), _raw_stream(device)))
    return q_out, k_out


def cp_qk_norm_rope_bwd(q, k, positions, dq_out, dk_out, q_weight=None, k_weight=None,
                        eps: float = 1e-6, theta: float = 10000.0,
                        rot_dim: Optional[int] = None, sections: Optional[Sequence[int]] = None,
                        interleaved: bool = False, inv_freq: Optional[Sequence[float]] = None):
    """Gradient of :func:`cp_qk_norm_rope_fwd` (same arguments, and the
    gradients of its outputs: contiguous, q's dtype).  Returns ``(dq, dk,
    dq_weight, dk_weight)``: dq, dk contiguous in q's dtype; the weight
    gradients fp32 ``[d]``, or None for a weight that is None."""
    f = _prepare(q, k, positions, q_weight, k_weight, eps, theta, rot_dim, sections,
                 interleaved, inv_freq)
    for g, x in ((dq_out, q), (dk_out, k)):
        if g.shape != x.shape or g.dtype != x.dtype or g.device != x.device or \
                not g.is_contiguous():
            raise CpError(2, "output gradients must be contiguous and match q and k")
    return _launch_bwd(f, q, k, positions, dq_out, dk_out, q_weight, k_weight)


def _launch_bwd(f, q, k, positions, dq_out, dk_out, q_weight, k_weight):
    device, d = q.device, q.shape[2]
    dq = torch.empty(q.shape, dtype=q.dtype, device=device)
    dk = torch.empty(k.shape, dtype=k.dtype, device=device)
    dqw, dkw = (None if w is None else torch.empty(d, dtype=torch.float32, device=device)
                for w in (q_weight, k_weight))
    lib = _b.lib()
    with _on_device(device):
        ws, nbytes = None, 0
        if dqw is not None or dkw is not None:
            nbytes = lib.cp_qk_norm_rope_bwd_workspace_size(f)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _b.check(lib.cp_qk_norm_rope_bwd(
            f, q.data_ptr(), k.data_ptr(), positions.data_ptr(), _at(q_weight), _at(k_weight),
            dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(), dk.data_ptr(), _at(dqw),
            _at(dkw), _at(ws), nbytes, _raw_stream(device)))
    return dq, dk, dqw, dkw
