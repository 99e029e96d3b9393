"""Attention with modified scores: a tanh cap, a bias by distance (slopes, or a
learned bias by bucket with its gradient), and an image prefix that attends to
itself in both directions.

Plans, tensor checks and workspaces for ``cp_attn_scored_fwd`` /
``cp_attn_scored_bwd`` (``include/cpattn.h``);
:func:`vlm_zigzag_head_gb300.autograd.cp_attention_scored` is the differentiable form.
"""
from __future__ import annotations

import array
import ctypes
import math
import numbers
from typing import List, Optional, Sequence, Union

import torch

from . import CP_BF16, CpError, Workspace, _binding as _b, _dt, _need_cuda
from .norm_rope import _at, _on_device, _raw_stream


def relative_buckets(n_buckets: int, max_distance: int) -> List[int]:
    """Bucket of every distance 0 .. ``max_distance``: one each below ``n_buckets //
    2``, then by the logarithm of the distance, the last bucket from ``max_distance`` on."""
    exact = n_buckets // 2
    if n_buckets < 2 or max_distance <= exact:
        raise CpError(1, "relative_buckets needs n_buckets >= 2 and max_distance > n_buckets / 2")
    span = math.log(max_distance / exact)

    def bucket(dist):
        ratio = math.log(dist / exact) / span
        # the nudge keeps exact powers, whose quotient may fall just short, in their bucket
        return min(n_buckets - 1, exact + int(ratio * (n_buckets - exact) + 1e-9))
    out = list(range(exact))
    for b in range(exact, n_buckets):   # its distances: up to the first one of the next bucket
        end = max_distance + 1
        if b < n_buckets - 1:
            end = min(end, int(exact * math.exp(span * (b + 1 - exact) / (n_buckets - exact))))
            while end > len(out) and bucket(end - 1) > b:
                end -= 1
            while end <= max_distance and bucket(end) <= b:
                end += 1
        out += [b] * (end - len(out))
    return out


class ScorePlan:
    """Work lists of :func:`cp_attn_scored_fwd` / :func:`cp_attn_scored_bwd` for one packing.

    ``cu_seqlens``: bounds of the packed samples ``[prefix_i ++ text_i]`` (any lengths).
    ``heads``: query heads.  ``prefix_len``: image tokens at the head of every sample (one
    number, or one per sample); with ``bidirectional_prefix`` they all see one another.
    ``rel_buckets``: bucket of each distance from 0 on, for a learned bias
    (:func:`relative_buckets`).

    Make it once per packing, outside stream capture (it copies the lists to the
    device and waits); every layer, stream and captured graph may share it.  A
    graph that was captured with it needs it alive.
    """

    def __init__(self, cu_seqlens: Sequence[int], heads: int,
                 prefix_len: Union[int, Sequence[int]] = 0, bidirectional_prefix: bool = False,
                 rel_buckets: Optional[Sequence[int]] = None, device="cuda"):
        device = torch.device(device)
        if device.type != "cuda":
            raise CpError(1, "a plan lives on a CUDA device")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        if torch.cuda.is_current_stream_capturing():
            raise CpError(1, "make the plan before the capture")
        if rel_buckets is not None:
            rel_buckets = list(rel_buckets)
            if not rel_buckets:
                raise CpError(1, "rel_buckets is empty")
        sms = torch.cuda.get_device_properties(device).multi_processor_count
        self.host, self.T = build_plan(cu_seqlens, heads, prefix_len, bidirectional_prefix,
                                       rel_buckets, sms)
        self.heads = int(heads)
        with torch.cuda.device(device):
            # a blocking copy: the lists are on the device before any stream uses them
            self.dev = torch.frombuffer(self.host, dtype=torch.uint8).to(device)
            self._stream = _raw_stream(device)
        self.device = device
        self._at = self.dev.data_ptr()
        self._block = (ctypes.c_char * len(self.host)).from_buffer(self.host)
        self._sizes = {}   # workspace bytes by dtypes, KV heads, head size and scale

    def _use(self, stream: int):
        """The device copy, kept from reuse until ``stream``, the current one, is done with it."""
        if stream != self._stream and not torch.cuda.is_current_stream_capturing():
            self.dev.record_stream(torch.cuda.current_stream(self.device))
        return self._at

    def _workspace_bytes(self, *shape):
        """Of the forward (dtype, KV heads, head size, scale), or with the gradients'
        dtype as a fifth of the backward."""
        if shape not in self._sizes:
            L = _b.lib()
            size = L.cp_attn_scored_bwd_workspace_size if len(shape) == 5 else \
                L.cp_attn_scored_fwd_workspace_size
            self._sizes[shape] = size(self._block, *shape)
        return self._sizes[shape]


def build_plan(cu_seqlens, heads, prefix_len, bidirectional_prefix, rel_buckets, n_sms):
    """Host block of a plan and its token count (needs no GPU)."""
    cu = _b.cu_array(cu_seqlens)
    n = len(cu_seqlens) - 1
    if n < 1:
        raise CpError(1, "cu_seqlens needs at least two entries")
    one = isinstance(prefix_len, numbers.Integral)
    lens = [int(prefix_len)] * n if one else [int(x) for x in prefix_len]
    if len(lens) != n:
        raise CpError(2, "prefix_len needs one entry per sample")
    pre = _b.cu_array(lens)
    nb = len(rel_buckets) if rel_buckets else 0
    buckets = None
    if nb:
        try:   # array copies whole numbers of any kind several times faster than ctypes
            buckets = (ctypes.c_int32 * nb).from_buffer(array.array("i", rel_buckets))
        except (TypeError, OverflowError):
            raise CpError(1, "rel_buckets must be whole numbers of 32 bits") from None
    args = (cu, n, pre, int(bool(bidirectional_prefix)), int(heads), int(n_sms), buckets, nb)
    size = _b.lib().cp_score_plan_size(*args)
    if size == 0:
        raise CpError(2, _b.lib().cp_last_error().decode(errors="replace"))
    host = bytearray(size)
    block = (ctypes.c_char * size).from_buffer(host)
    _b.check(_b.lib().cp_score_plan_build(*args, block, size))
    return host, int(cu[n])


def _scores(q, softcap, slopes, rel_bias):
    s = _b.ScoreDesc()
    s.softcap = float(softcap)
    H = q.shape[1]
    if slopes is not None:
        if slopes.shape != (H,) or slopes.dtype != torch.float32 or not slopes.is_contiguous() \
                or slopes.device != q.device:
            raise CpError(2, "slopes must be a contiguous fp32 [H] tensor on q's device")
        s.slopes = slopes.data_ptr()
    if rel_bias is not None:
        if rel_bias.dim() != 2 or rel_bias.shape[0] != H or rel_bias.device != q.device:
            raise CpError(2, "rel_bias must be [H, n_buckets] on q's device")
        s.rel_bias = rel_bias.data_ptr()
        s.bias_dtype = _dt(rel_bias)
        s.bias_stride_h, s.bias_stride_b = rel_bias.stride()
        s.n_buckets = rel_bias.shape[1]
    return s


def _check(q, k, v, plan):
    if q.dim() != 3 or k.dim() != 3 or v.shape != k.shape:
        raise CpError(2, "q must be [T, H, d]; k and v [T, H_kv, d]")
    if k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
        raise CpError(2, "q, k and v must share tokens and head size")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise CpError(3, "q, k and v must share a dtype")
    if any(t.device != plan.device for t in (q, k, v)):
        raise CpError(1, "q, k, v and the plan must share a device")


def _like(t, shape, dtype, device, name):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device:
        raise CpError(2, "%s has another shape, dtype or device" % name)


def _space(workspace, nbytes, device):
    """(holder, pointer, bytes): the caller's workspace, or a new one for this call alone."""
    if workspace is None:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return buf, buf.data_ptr(), nbytes
    workspace.get(nbytes, device)
    return workspace, workspace.ptr(), workspace.nbytes()


def cp_attn_scored_fwd(q, k, v, plan: ScorePlan, softmax_scale: float, softcap: float = 0.0,
                       slopes=None, rel_bias=None, out=None, lse=None,
                       workspace: Optional[Workspace] = None, residual: bool = False,
                       out_lo=None):
    """Packed causal attention whose scores are capped (``softcap``), get a bias
    ``-slopes[h] * distance`` or ``rel_bias[h, bucket(distance)]``, or both; returns ``(out,
    lse)`` as :func:`cp_attn_fwd`, and with ``residual=True`` (bf16) also the rounding
    remainder of out for :func:`cp_attn_scored_bwd`.

    ``q [T,H,d]``, ``k``/``v [T,H_kv,d]`` contiguous bf16 or fp32; ``slopes [H]`` fp32;
    ``rel_bias [H, n_buckets]`` bf16 or fp32, any strides.  Without ``workspace`` each
    call takes one of its own, so calls on several streams may overlap."""
    _need_cuda(q, k, v, out, lse, out_lo)
    _check(q, k, v, plan)
    T, H, _ = q.shape
    if out is not None:
        _like(out, q.shape, q.dtype, q.device, "out")
    if lse is not None:
        _like(lse, (H, T), torch.float32, q.device, "lse")
    if out_lo is not None:
        _like(out_lo, q.shape, q.dtype, q.device, "out_lo")
    s = _scores(q, softcap, slopes, rel_bias)
    return _launch_fwd(s, q, k, v, plan, float(softmax_scale), out, lse, workspace, residual,
                       out_lo)


def _launch_fwd(s, q, k, v, plan, scale, out=None, lse=None, workspace=None, residual=False,
                out_lo=None):
    """The forward on checked tensors."""
    T, H, d = q.shape
    H_kv, device, dt = k.shape[1], q.device, _dt(q)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=device)
    if lse is None:
        lse = torch.empty((H, T), dtype=torch.float32, device=device)
    if out_lo is None and residual and dt == CP_BF16:
        out_lo = torch.empty(q.shape, dtype=q.dtype, device=device)
    with _on_device(device):
        ws, ptr, size = _space(workspace, plan._workspace_bytes(dt, H_kv, d, scale), device)
        stream = _raw_stream(device)
        _b.check(_b.lib().cp_attn_scored_fwd(
            plan._block, plan._use(stream), q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, T, H,
            H_kv, d, s, scale, out.data_ptr(), lse.data_ptr(), _at(out_lo), ptr, size, stream))
    return (out, lse, out_lo) if residual else (out, lse)


def cp_attn_scored_bwd(q, k, v, out, lse, dout, plan: ScorePlan, softmax_scale: float,
                       softcap: float = 0.0, slopes=None, rel_bias=None,
                       workspace: Optional[Workspace] = None, grads=None, out_lo=None,
                       grad_dtype=torch.float32):
    """Gradient of :func:`cp_attn_scored_fwd`: ``(dq, dk, dv)``, and with ``rel_bias`` a
    fourth, ``dbias [H, n_buckets]``.  ``grad_dtype``: fp32, or bf16 for bf16 inputs
    (dbias is then in rel_bias's dtype).  ``grads`` may supply dq, dk, dv."""
    _need_cuda(q, k, v, out, lse, dout, out_lo, *(grads or ()))
    _check(q, k, v, plan)
    T, H, _ = q.shape
    for t, name in ((out, "out"), (dout, "dout"), (out_lo, "out_lo")):
        if t is not None:
            _like(t, q.shape, q.dtype, q.device, name)
    _like(lse, (H, T), torch.float32, q.device, "lse")
    for t, x, name in zip(grads or (), (q, k, v), ("dq", "dk", "dv")):
        _like(t, x.shape, grad_dtype, q.device, name)
    s = _scores(q, softcap, slopes, rel_bias)
    got = _launch_bwd(s, q, k, v, out, lse, dout, plan, float(softmax_scale), rel_bias,
                      workspace, grads, out_lo, grad_dtype)
    return got if rel_bias is not None else got[:3]


def _launch_bwd(s, q, k, v, out, lse, dout, plan, scale, rel_bias, workspace, grads, out_lo,
                grad_dtype):
    """The backward on checked tensors; dbias is None without a bias."""
    T, H, d = q.shape
    H_kv, device, dt = k.shape[1], q.device, _dt(q)
    dq, dk, dv = grads or (torch.empty(x.shape, dtype=grad_dtype, device=device)
                           for x in (q, k, v))
    gdt = bdt = _dt(dq)
    dbias = None
    if rel_bias is not None:
        dbias = torch.empty(rel_bias.shape, device=device, dtype=torch.float32
                            if grad_dtype == torch.float32 else rel_bias.dtype)
        bdt = _dt(dbias)
    with _on_device(device):
        ws, ptr, size = _space(workspace, plan._workspace_bytes(dt, H_kv, d, scale, gdt), device)
        stream = _raw_stream(device)
        _b.check(_b.lib().cp_attn_scored_bwd(
            plan._block, plan._use(stream), q.data_ptr(), k.data_ptr(), v.data_ptr(),
            out.data_ptr(), _at(out_lo), lse.data_ptr(), dout.data_ptr(), dt, T, H, H_kv, d, s,
            scale, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), gdt, _at(dbias), bdt, ptr, size,
            stream))
    return dq, dk, dv, dbias
