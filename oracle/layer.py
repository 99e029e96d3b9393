"""fp64 oracle of the operators around the attention of a transformer layer: layer
norm, rotation of heads, and the gated feed-forward block, with their gradients.
Written from the formulas; no code is shared with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

from .scored import _f64, _rotate, rope_matrix_parts


def layer_norm_fwd(x, weight, bias, eps):
    """(y, mean, rstd) of rows ``[T, D]``."""
    x = _f64(x)
    mean = x.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    y = (x - mean) * rstd
    if weight is not None:
        y = y * _f64(weight)
    if bias is not None:
        y = y + _f64(bias)
    return y, mean[..., 0], rstd[..., 0]


def layer_norm_bwd(x, dy, weight, eps):
    """(dx, dweight, dbias)."""
    x, dy = _f64(x), _f64(dy)
    n, _, rstd = layer_norm_fwd(x, None, None, eps)
    g = dy if weight is None else dy * _f64(weight)
    dx = rstd[..., None] * (g - g.mean(-1, keepdims=True) - n * (g * n).mean(-1, keepdims=True))
    return dx, (dy * n).sum(0), dy.sum(0)


def rope(x, positions, rot_dim, inv_freq, sections, interleaved, amplitude=1.0, sign=1.0):
    """The rotation (sign 1) or its gradient (sign -1) of ``[T, heads, d]``."""
    x = _f64(x)
    i, j, angle = rope_matrix_parts(positions, rot_dim, inv_freq, sections, interleaved)
    y = _rotate(x, i, j, angle, sign)
    y[..., :rot_dim] *= amplitude
    return y


_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(g, act):
    """The activation and its derivative."""
    if act == "silu":
        s = 0.5 * (1 + np.tanh(0.5 * g))
        return g * s, s + g * s * (1 - s)
    if act == "gelu":
        c = 0.5 * (1 + _erf(g / math.sqrt(2)))
        return g * c, c + g * np.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = np.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 0.134145 * g * g)


def gated_ffn(x, w_gate, w_up, w_down, act, dy=None):
    """y, and with dy ``(y, dx, dw_gate, dw_up, dw_down)``: y = (act(x Wg^T) (x Wu^T)) Wd^T."""
    x, wg, wu, wd = _f64(x), _f64(w_gate), _f64(w_up), _f64(w_down)
    g, u = x @ wg.T, x @ wu.T
    a, da = activation(g, act)
    y = (a * u) @ wd.T
    if dy is None:
        return y
    dy = _f64(dy)
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    return y, dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ (a * u)
