"""Rotation of query and key heads by their positions, and its gradient.

Tensor checks and descriptors for ``cp_rope_fwd`` / ``cp_rope_bwd``
(``include/cpattn.h``), and the frequencies of contexts longer than those a model was
trained on; :func:`vlm_zigzag_head_gb300.autograd.rope` is the differentiable form.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Sequence, Tuple

import torch

from . import CpError, _binding as _b, _dt
from .norm_rope import _check_heads, _on_device, _raw_stream, _wants_grad


class Frequencies(tuple):
    """Floats, one a rotated pair: what :func:`rope_frequencies` returns (a call takes them as
    they are, where it converts each entry of another sequence)."""


def rope_frequencies(rot_dim: int, theta: float = 10000.0, *, scaling: str = "none",
                     factor: float = 1.0, trained_length: int = 8192, low: float = 1.0,
                     high: float = 32.0) -> Tuple[float, ...]:
    """Radians per position of every rotated pair, for ``inv_freq``.

    f_p = theta ** (-2 p / rot_dim), scaled for a context ``factor`` times as long as the
    ``trained_length`` tokens a model was trained on:

    * ``"none"``;
    * ``"linear"``: f_p / factor (positions are interpolated);
    * ``"base"``: theta times factor ** (rot_dim / (rot_dim - 2)), so that the slowest pair
      is interpolated and the fastest one stays;
    * ``"by_parts"``: a pair that turns more than ``high`` times within the trained length
      stays, one that turns less than ``low`` times is interpolated, and between the two
      the share that stays grows linearly with the turns.  It usually goes with an
      amplitude of ``1 + 0.1 * log(factor)``."""
    if rot_dim < 0 or rot_dim % 2:
        raise CpError(2, "rot_dim must be even")
    if not theta > 0 or not factor > 0:
        raise CpError(1, "theta and factor must be positive")
    if scaling == "base":
        if rot_dim <= 2:
            raise CpError(2, "scaling the base needs more than one pair")
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    freq = [theta ** (-2.0 * p / rot_dim) for p in range(rot_dim // 2)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "by_parts":
        if not high > low or trained_length < 1:
            raise CpError(1, "by_parts needs high > low and a trained length")
        out = []
        for f in freq:
            turns = f * trained_length / (2 * math.pi)
            stays = min(1.0, max(0.0, (turns - low) / (high - low)))
            out.append(f * (stays + (1 - stays) / factor))
        freq = out
    elif scaling not in ("none", "base"):
        raise CpError(1, "scaling must be none, linear, base or by_parts")
    return Frequencies(freq)


@functools.lru_cache(maxsize=256)
def _desc(dtype, q_shape, q_stride, k_shape, k_stride, pos_shape, theta, rot_dim, sections,
          interleaved, inv_freq, amplitude, inplace):
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
        inv_freq = rope_frequencies(rot, theta)
    elif len(inv_freq) != rot // 2:
        raise CpError(2, "inv_freq must have rot_dim / 2 entries")
    f = _b.RopeDesc()
    f.dtype = dtype
    f.T, f.H, f.H_kv, f.d = T, H, k_shape[1], d
    # the stride of a dimension of one element is never used
    f.q_stride_t, f.q_stride_h = (s if n > 1 else 0 for s, n in zip(q_stride, q_shape[:2]))
    f.k_stride_t, f.k_stride_h = (s if n > 1 else 0 for s, n in zip(k_stride, k_shape[:2]))
    if inplace:
        for stride, shape, name in ((q_stride, q_shape, "q"), (k_stride, k_shape, "k")):
            if T > 0 and not _rows_apart(stride, shape):
                raise CpError(1, "%s shares memory between its heads: not in place" % name)
        f.q_out_stride_t, f.q_out_stride_h = f.q_stride_t, f.q_stride_h
        f.k_out_stride_t, f.k_out_stride_h = f.k_stride_t, f.k_stride_h
    else:
        f.q_out_stride_t, f.q_out_stride_h = H * d, d
        f.k_out_stride_t, f.k_out_stride_h = k_shape[1] * d, d
    f.rot_dim, f.interleaved, f.n_axes = rot, int(interleaved), axes
    for i, n in enumerate(sections):
        f.sections[i] = n
    f.inv_freq = (ctypes.c_double * max(1, len(inv_freq)))(*inv_freq)
    f.amplitude = amplitude
    return f


def _rows_apart(stride, shape):
    """Whether no two heads of a ``[T, heads, d]`` view overlap (dimensions nested by stride)."""
    room = shape[2]
    for s, n in sorted((s, n) for s, n in zip(stride[:2], shape[:2]) if n > 1):
        if s < room:
            return False
        room = s * n
    return True


def _disjoint(q, k):
    """Whether q and k, neither overlapping itself, share no element."""
    size = q.element_size()

    def span(x):
        return x.data_ptr(), x.data_ptr() + size * (
            1 + sum((n - 1) * s for n, s in zip(x.shape, x.stride())))
    (qa, qb), (ka, kb) = span(q), span(k)
    if qb <= ka or kb <= qa:
        return True
    # interleaved slices of one buffer: the same token stride, and within it each its own part
    step = q.stride(0) * size
    if q.stride(0) != k.stride(0) or step == 0 or (ka - qa) % size:
        return False
    q_len, k_len = ((x.shape[1] - 1) * x.stride(1) * size + x.shape[2] * size for x in (q, k))
    gap = (ka - qa) % step
    return q_len <= gap and gap + k_len <= step


def _prepare(q, k, positions, theta, rot_dim, sections, interleaved, inv_freq, amplitude,
             inplace=False):
    if inplace and _wants_grad(q, k):   # a graph would go on as if nothing had happened
        raise CpError(1, "q or k is being differentiated: not in place (autograd.rope rotates out "
                         "of place; detached tensors and no_grad leave the graph)")
    _check_heads(q, "q")
    _check_heads(k, "k", q)
    if positions.dtype != torch.int32 or positions.device != q.device or \
            not positions.is_contiguous():
        raise CpError(3, "positions must be a contiguous int32 tensor on q's device")
    f = _desc(_dt(q), tuple(q.shape), q.stride(), tuple(k.shape), k.stride(),
              tuple(positions.shape), float(theta), rot_dim,
              None if sections is None else tuple(int(n) for n in sections), bool(interleaved),
              inv_freq if inv_freq is None or type(inv_freq) is Frequencies else
              Frequencies(float(x) for x in inv_freq), float(amplitude), bool(inplace))
    if inplace and f.T > 0 and not _disjoint(q, k):
        raise CpError(1, "q and k share memory: not in place")
    return f


def cp_rope_fwd(q, k, positions, *, theta: float = 10000.0, rot_dim: Optional[int] = None,
                sections: Optional[Sequence[int]] = None, interleaved: bool = False,
                inv_freq: Optional[Sequence[float]] = None, amplitude: float = 1.0,
                inplace: bool = False):
    """Rotate every head of ``q [T,H,d]`` and ``k [T,H_kv,d]`` (bf16 or fp32; any token and
    head strides, e.g. slices of one projection's output) by its position.

    ``positions``, ``rot_dim``, ``sections``, ``interleaved`` and ``inv_freq`` as in
    :func:`cp_qk_norm_rope_fwd`; :func:`rope_frequencies` gives ``inv_freq`` for long
    contexts.  ``amplitude`` multiplies the rotated elements; the others are copied.
    Returns contiguous ``(q_out, k_out)``, or with ``inplace`` q and k themselves, written
    over: refused where autograd would have to know of it (q or k requires grad while gradients
    are recorded, or carries a forward-mode tangent)."""
    f = _prepare(q, k, positions, theta, rot_dim, sections, interleaved, inv_freq, amplitude,
                 inplace)
    return _launch(_b.lib().cp_rope_fwd, f, q, k, positions, inplace)


def cp_rope_bwd(dq_out, dk_out, positions, *, theta: float = 10000.0,
                rot_dim: Optional[int] = None, sections: Optional[Sequence[int]] = None,
                interleaved: bool = False, inv_freq: Optional[Sequence[float]] = None,
                amplitude: float = 1.0, inplace: bool = False):
    """Gradient of :func:`cp_rope_fwd` (same options; the gradients of its outputs, any token
    and head strides).  Returns contiguous ``(dq, dk)``, or with ``inplace`` its arguments,
    written over (refused as in :func:`cp_rope_fwd`)."""
    f = _prepare(dq_out, dk_out, positions, theta, rot_dim, sections, interleaved, inv_freq,
                 amplitude, inplace)
    return _launch(_b.lib().cp_rope_bwd, f, dq_out, dk_out, positions, inplace)


def _launch(entry, f, q, k, positions, inplace=False):
    device = q.device
    if inplace:
        q_out, k_out = q, k
    else:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=device)
        k_out = torch.empty(k.shape, dtype=k.dtype, device=device)
    with _on_device(device):
        _b.check(entry(f, q.data_ptr(), k.data_ptr(), positions.data_ptr(), q_out.data_ptr(),
                       k_out.data_ptr(), _raw_stream(device)))
    if inplace:   # a graph that saved them for its backward must notice
        for x in (q, k):
            if not x.is_inference():
                torch.autograd.graph.increment_version(x)
    return q_out, k_out
