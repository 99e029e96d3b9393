"""torch.autograd binding of context-parallel causal attention.

The multimodal context-parallel page (§4.2, gradient path; §5.2, the image
prefix) has every CP rank differentiate its own text queries against the
replicated image prefix, then sums those per-rank prefix gradients with an
AllReduce hooked onto the image embeddings' gradient.  Here every rank lives
in one GPU's memory: ``cp_attn_bwd`` sums the per-rank prefix terms in a fixed
order (ranks 0..P-1, then the prefix queries' own term) before it returns, so
the gradients that reach autograd are already the reduced ones.

``prefix_hook`` gives a caller the quantity the page's hook reduces.  It is
called during the backward with the per-rank terms ``[2, P+1, n*N, H_kv, d]``
(dK, dV; slot P is the prefix queries' own term), before autograd receives
the summed gradients.

Every step runs in the library's CUDA kernels; this module only marshals
tensors through :mod:`torch.autograd`.
"""
from __future__ import annotations

from typing import Callable, Optional, Sequence

import torch
from torch.autograd.function import once_differentiable

from . import CpError, ScorePlan, Workspace, cp_attn_bwd, cp_attn_fwd, norm_rope, scored
from . import _binding as _b
from . import ffn as _ffn
from . import layer_norm as _layer_norm
from . import rope as _rope
from .norm_rope import _wants_grad


class CPAttention(torch.autograd.Function):
    """``(out, lse) = CPAttention.apply(q, k, v, cu_seqlens, P, prefix_len,
    softmax_scale, prefix_hook)``.  lse is not differentiable."""

    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, P, prefix_len, softmax_scale, prefix_hook):
        cu = tuple(int(x) for x in cu_seqlens)
        if q.dtype == torch.bfloat16:
            # the bf16 remainder of the output keeps D = dO.O exact in the backward
            out, lse, out_lo = cp_attn_fwd(q, k, v, cu, P, prefix_len, softmax_scale,
                                           residual=True)
        else:
            out, lse = cp_attn_fwd(q, k, v, cu, P, prefix_len, softmax_scale)
            out_lo = None
        ctx.save_for_backward(q, k, v, out, lse, out_lo)
        ctx.meta = (cu, int(P), int(prefix_len), float(softmax_scale), prefix_hook)
        ctx.mark_non_differentiable(lse)
        return out, lse

    @staticmethod
    def backward(ctx, dout, _dlse):
        q, k, v, out, lse, out_lo = ctx.saved_tensors
        cu, P, N, scale, hook = ctx.meta
        if dout is None:
            dout = torch.zeros_like(out)
        dout = dout.to(q.dtype).contiguous()
        want_pre = hook is not None and N > 0
        res = cp_attn_bwd(q, k, v, out, lse, dout, cu, P, N, scale,
                          per_rank_prefix=want_pre, out_lo=out_lo)
        dq, dk, dv = res[:3]
        if want_pre:
            hook(res[3])
        grads = []
        for g, x, need in zip((dq, dk, dv), (q, k, v), ctx.needs_input_grad[:3]):
            grads.append(g.to(x.dtype) if need else None)
        return (*grads, None, None, None, None, None)


def cp_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                 cu_seqlens: Sequence[int], P: int, prefix_len: int = 0,
                 softmax_scale: Optional[float] = None,
                 prefix_hook: Optional[Callable[[torch.Tensor], None]] = None):
    """Differentiable zigzag context-parallel causal attention over packed
    samples ``[prefix_i ++ text_i]`` (THD layout ``[T, H, d]``, bf16 or fp32,
    on a CUDA device).  Returns ``(out, lse)``; gradients flow to q, k and v.
    ``k`` / ``v`` may hold fewer heads than ``q`` (grouped-query attention:
    query head h reads KV head h // (H / H_kv)).  ``softmax_scale`` defaults
    to ``1/sqrt(d)``."""
    if softmax_scale is None:
        softmax_scale = q.shape[-1] ** -0.5
    return CPAttention.apply(q, k, v, cu_seqlens, P, prefix_len, softmax_scale, prefix_hook)


def _dense(x: torch.Tensor) -> torch.Tensor:
    """A contiguous, 16-byte aligned tensor (a copy of any other view)."""
    x = x.contiguous()
    return x if x.data_ptr() % 16 == 0 else x.clone()


class QKNormRope(torch.autograd.Function):
    """``(q_out, k_out) = QKNormRope.apply(q, k, positions, q_weight, k_weight, desc, options)``."""

    @staticmethod
    def forward(ctx, q, k, positions, q_weight, k_weight, desc, options):
        ctx.save_for_backward(q, k, positions, q_weight, k_weight)
        ctx.meta = (desc, options, q.stride(), k.stride())
        ctx.set_materialize_grads(False)
        return norm_rope._launch_fwd(desc, q, k, positions, q_weight, k_weight)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, positions, q_weight, k_weight = ctx.saved_tensors
        need = ctx.needs_input_grad
        desc, options, q_stride, k_stride = ctx.meta
        # saved tensors may come back with other strides (offloaded, recomputed)
        if q.stride() != q_stride or k.stride() != k_stride:
            desc = norm_rope._prepare(q, k, positions, q_weight, k_weight, *options)
        # an output that nothing used has no gradient
        dq_out = torch.zeros_like(q, memory_format=torch.contiguous_format) if dq_out is None \
            else _dense(dq_out)
        dk_out = torch.zeros_like(k, memory_format=torch.contiguous_format) if dk_out is None \
            else _dense(dk_out)
        dq, dk, dqw, dkw = norm_rope._launch_bwd(desc, q, k, positions, dq_out, dk_out, q_weight,
                                                 k_weight)
        return (dq if need[0] else None, dk if need[1] else None, None,
                dqw.to(q_weight.dtype) if need[3] else None,
                dkw.to(k_weight.dtype) if need[4] else None, None, None)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor,
                 q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                 theta: float = 10000.0, rot_dim: Optional[int] = None,
                 sections: Optional[Sequence[int]] = None, interleaved: bool = False,
                 inv_freq: Optional[Sequence[float]] = None):
    """Differentiable :func:`~vlm_zigzag_head_gb300.cp_qk_norm_rope_fwd`: RMS norm of every head of q and k
    and the position rotation, in one pass.  Returns contiguous ``(q_out, k_out)``,
    ready for :func:`cp_attention`; gradients flow to q, k and the weights (backward only:
    forward mode raises).  To capture the backward into a graph, call
    :func:`~vlm_zigzag_head_gb300.cp_qk_norm_rope_bwd`, which involves no leaves."""
    sections = None if sections is None else tuple(sections)
    inv_freq = None if inv_freq is None else tuple(inv_freq)
    options = (eps, theta, rot_dim, sections, interleaved, inv_freq)
    desc = norm_rope._prepare(q, k, positions, q_weight, k_weight, *options)
    if not _wants_grad(q, k, q_weight, k_weight):
        return norm_rope._launch_fwd(desc, q, k, positions, q_weight, k_weight)
    return QKNormRope.apply(q, k, positions, q_weight, k_weight, desc, options)


class Rope(torch.autograd.Function):
    """``(q_out, k_out) = Rope.apply(q, k, positions, desc, options)``."""

    @staticmethod
    def forward(ctx, q, k, positions, desc, options):
        ctx.save_for_backward(positions)
        ctx.meta = options, q.shape, k.shape, q.dtype
        ctx.set_materialize_grads(False)
        return _rope._launch(_b.lib().cp_rope_fwd, desc, q, k, positions)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        positions, = ctx.saved_tensors
        options, q_shape, k_shape, dtype = ctx.meta
        if dq_out is None and dk_out is None:
            return (None,) * 5
        # an output that nothing used has no gradient
        dq_out, dk_out = (torch.zeros(shape, dtype=dtype, device=positions.device) if g is None
                          else g if g.stride(-1) == 1 else g.contiguous()
                          for g, shape in ((dq_out, q_shape), (dk_out, k_shape)))
        desc = _rope._prepare(dq_out, dk_out, positions, *options)
        dq, dk = _rope._launch(_b.lib().cp_rope_bwd, desc, dq_out, dk_out, positions)
        need = ctx.needs_input_grad
        return dq if need[0] else None, dk if need[1] else None, None, None, None


def rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, *, theta: float = 10000.0,
         rot_dim: Optional[int] = None, sections: Optional[Sequence[int]] = None,
         interleaved: bool = False, inv_freq: Optional[Sequence[float]] = None,
         amplitude: float = 1.0):
    """Differentiable :func:`~vlm_zigzag_head_gb300.cp_rope_fwd`: every head of q and k turned by
    its position.  Returns contiguous ``(q_out, k_out)``, ready for :func:`cp_attention`;
    gradients flow to q and k (backward only: forward mode raises).  To capture the backward
    into a graph, call :func:`~vlm_zigzag_head_gb300.cp_rope_bwd`, which involves no leaves."""
    options = (theta, rot_dim, None if sections is None else tuple(sections), interleaved,
               inv_freq if inv_freq is None else _rope.Frequencies(float(f) for f in inv_freq),
               amplitude)
    desc = _rope._prepare(q, k, positions, *options)
    if not _wants_grad(q, k):
        return _rope._launch(_b.lib().cp_rope_fwd, desc, q, k, positions)
    return Rope.apply(q, k, positions, desc, options)


class LayerNorm(torch.autograd.Function):
    """``y = LayerNorm.apply(x, weight, bias, eps)``."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        rows = _layer_norm._rows(x, "x")
        desc = _layer_norm._prepare(rows, weight, bias, eps)
        y, mean, rstd = _layer_norm._launch_fwd(desc, rows, weight, bias, x.shape)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        ctx.set_materialize_grads(False)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        if dy is None:   # what used y has no gradient for it
            return (None,) * 4
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = _layer_norm.cp_layer_norm_bwd(x, dy, mean, rstd, weight, input_grad=need[0],
                                                   weight_grad=need[1], bias_grad=need[2])
        return (dx, dw.to(weight.dtype) if need[1] else None,
                db.to(ctx.bias_dtype) if need[2] else None, None)


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5):
    """Differentiable :func:`~vlm_zigzag_head_gb300.cp_layer_norm_fwd` of the last dimension of
    ``x [..., D]``.  Returns y, contiguous; gradients flow to x, weight and bias (backward
    only: forward mode raises).  To capture the backward into a graph, call
    :func:`~vlm_zigzag_head_gb300.cp_layer_norm_bwd`, which involves no leaves."""
    if not _wants_grad(x, weight, bias):
        rows = _layer_norm._rows(x, "x")
        desc = _layer_norm._prepare(rows, weight, bias, eps)
        return _layer_norm._launch_fwd(desc, rows, weight, bias, x.shape, stats=False)[0]
    return LayerNorm.apply(x, weight, bias, eps)


class GatedFfn(torch.autograd.Function):
    """``y = GatedFfn.apply(x, w_gate, w_up, w_down, activation, workspace)`` on 16-byte aligned
    rows."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, activation, workspace):
        y, gate, up = _ffn.cp_gated_ffn_fwd(x, w_gate, w_up, w_down, activation, keep=True,
                                            workspace=workspace)
        ctx.save_for_backward(x, w_gate, w_up, w_down, gate, up)
        ctx.activation, ctx.workspace = activation, workspace
        ctx.set_materialize_grads(False)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        if dy is None:   # what used y has no gradient for it
            return (None,) * 6
        # saved tensors may come back elsewhere and with other strides (offloaded, recomputed)
        x, w_gate, w_up, w_down, gate, up = (_ffn._aligned(t) for t in ctx.saved_tensors)
        return (*_ffn.cp_gated_ffn_bwd(x, w_gate, w_up, w_down, gate, up, _ffn._aligned(dy),
                                       ctx.activation, grad_dtype=x.dtype,
                                       wanted=ctx.needs_input_grad[:4],
                                       workspace=ctx.workspace), None, None)


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, *,
              activation: str = "silu", workspace: Optional[Workspace] = None):
    """Differentiable :func:`~vlm_zigzag_head_gb300.cp_gated_ffn_fwd`: (a(x w_gate^T) * (x
    w_up^T)) w_down^T of the last dimension of ``x [..., D]``, with ``a`` one of ``"silu"``,
    ``"gelu"``, ``"gelu_tanh"``.  Tensors whose rows do not lie on 16-byte boundaries are
    copied.  Gradients flow to x and the weights (backward only: forward mode raises); a
    gradient that is not needed is not computed.  To capture the backward into a graph, call
    :func:`~vlm_zigzag_head_gb300.cp_gated_ffn_bwd`, which involves no leaves.

    With ``workspace`` both directions use it (their calls then belong on one stream), and
    :func:`~vlm_zigzag_head_gb300.cp_workspace_status` tells of the last of them whether a
    bounded device wait ran out, which leaves its results unwritten; without one nothing does."""
    x, w_gate, w_up, w_down = (_ffn._aligned(t) for t in (x, w_gate, w_up, w_down))
    if not _wants_grad(x, w_gate, w_up, w_down):
        return _ffn.cp_gated_ffn_fwd(x, w_gate, w_up, w_down, activation, workspace=workspace)
    return GatedFfn.apply(x, w_gate, w_up, w_down, activation, workspace)


class CPAttentionScored(torch.autograd.Function):
    """``(out, lse) = CPAttentionScored.apply(q, k, v, rel_bias, slopes, plan,
    softmax_scale, desc)`` on checked tensors.  lse and slopes are not differentiable."""

    @staticmethod
    def forward(ctx, q, k, v, rel_bias, slopes, plan, softmax_scale, desc):
        # the bf16 remainder of the output keeps D = dO.O exact in the backward
        out, lse, out_lo = scored._launch_fwd(desc, q, k, v, plan, softmax_scale, residual=True)
        ctx.save_for_backward(q, k, v, rel_bias, slopes, out, lse, out_lo)
        ctx.meta = (plan, softmax_scale, desc.softcap)
        ctx.set_materialize_grads(False)   # lse's would be zeros to fill; dout may be None
        ctx.mark_non_differentiable(lse)
        return out, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, _dlse):
        if dout is None:   # what used out has no gradient for it
            return (None,) * 8
        q, k, v, rel_bias, slopes, out, lse, out_lo = ctx.saved_tensors
        plan, scale, softcap = ctx.meta
        # saved tensors may come back elsewhere and with other strides (offloaded, recomputed)
        q, k, v, out, lse = (_dense(x) for x in (q, k, v, out, lse))
        out_lo = None if out_lo is None else _dense(out_lo)
        desc = scored._scores(q, softcap, slopes, rel_bias)
        got = scored._launch_bwd(desc, q, k, v, out, lse, _dense(dout), plan, scale, rel_bias,
                                 None, None, out_lo, q.dtype)
        need = ctx.needs_input_grad
        dbias = got[3].to(rel_bias.dtype) if need[3] else None
        return (*(g if n else None for g, n in zip(got[:3], need)), dbias, None, None, None, None)


def cp_attention_scored(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, plan: ScorePlan,
                        softmax_scale: Optional[float] = None, *, softcap: float = 0.0,
                        slopes: Optional[torch.Tensor] = None,
                        rel_bias: Optional[torch.Tensor] = None):
    """Differentiable packed causal attention with modified scores (see
    :func:`~vlm_zigzag_head_gb300.cp_attn_scored_fwd`): a tanh cap, a bias by distance, and the plan's
    bidirectional prefix.  q, k and v of any strides (copied where not contiguous).
    Returns ``(out, lse)``; gradients flow to q, k, v and ``rel_bias`` (backward only: forward
    mode raises).
    ``softmax_scale`` defaults to ``1/sqrt(d)``.  To capture the backward into a graph, call
    :func:`~vlm_zigzag_head_gb300.cp_attn_scored_bwd`, which involves no leaves."""
    if softmax_scale is None:
        softmax_scale = q.shape[-1] ** -0.5
    if slopes is not None and slopes.requires_grad:
        raise CpError(8, "slopes have no gradient here; a learned bias goes in rel_bias")
    if not (q.is_cuda and k.is_cuda and v.is_cuda):
        raise CpError(1, "tensors must live on a CUDA device")
    scored._check(q, k, v, plan)
    q, k, v = _dense(q), _dense(k), _dense(v)
    desc = scored._scores(q, softcap, slopes, rel_bias)
    if not _wants_grad(q, k, v, rel_bias, slopes):
        return scored._launch_fwd(desc, q, k, v, plan, float(softmax_scale))
    return CPAttentionScored.apply(q, k, v, rel_bias, slopes, plan, float(softmax_scale), desc)
