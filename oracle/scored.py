"""fp64 oracle of the query / key norm with rotation, and of attention with
modified scores (tanh cap, distance bias, learned bucket bias, a prefix that
attends to itself in both directions).  Written from the formulas, one sample
and one head at a time; no code is shared with the CUDA path.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Sequence

import numpy as np


def _f64(x):
    if hasattr(x, "detach"):
        import torch
        x = x.detach().to("cpu", torch.float64).numpy()
    return np.asarray(x, dtype=np.float64)


# --------------------------------------------------------------------------- norm and rotation
def rope_matrix_parts(positions, rot_dim: int, inv_freq: Sequence[float], sections: Sequence[int],
                      interleaved: bool):
    """Index pairs (i, j) and angles [T, rot_dim / 2] of the rotated elements."""
    pos = _f64(positions).reshape(len(sections), -1)
    pairs = rot_dim // 2
    p = np.arange(pairs)
    i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + pairs)
    axis = np.repeat(np.arange(len(sections)), sections)
    # whole turns drop out in extended precision, so far positions stay exact
    turns = pos[axis].T.astype(np.longdouble) * (np.asarray(inv_freq, np.longdouble) /
                                                 (2 * np.longdouble(np.pi)))
    angle = np.asarray((turns - np.floor(turns)) * 2 * np.pi, dtype=np.float64)
    return i, j, angle


def _rotate(z, i, j, angle, sign):
    y = z.copy()
    c, s = np.cos(angle)[:, None, :], sign * np.sin(angle)[:, None, :]
    y[..., i] = z[..., i] * c - z[..., j] * s
    y[..., j] = z[..., j] * c + z[..., i] * s
    return y


def norm_rope_fwd(x, positions, weight, eps, rot_dim, inv_freq, sections, interleaved):
    """y = R (x / rms(x) * w) for one of q, k: ``[T, heads, d]``."""
    x = _f64(x)
    w = np.ones(x.shape[-1]) if weight is None else _f64(weight)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    i, j, angle = rope_matrix_parts(positions, rot_dim, inv_freq, sections, interleaved)
    return _rotate(n * w, i, j, angle, 1.0)


def norm_rope_bwd(x, dy, positions, weight, eps, rot_dim, inv_freq, sections, interleaved):
    """(dx, dw) of :func:`norm_rope_fwd`."""
    x, dy = _f64(x), _f64(dy)
    w = np.ones(x.shape[-1]) if weight is None else _f64(weight)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    i, j, angle = rope_matrix_parts(positions, rot_dim, inv_freq, sections, interleaved)
    g = _rotate(dy, i, j, angle, -1.0)
    dw = (g * n).sum((0, 1))
    gw = g * w
    return r * (gw - n * (gw * n).mean(-1, keepdims=True)), dw


# --------------------------------------------------------------------------- attention
class Scores(NamedTuple):
    """What happens to the scaled products before the softmax."""
    softcap: float = 0.0                      # x -> softcap tanh(x / softcap); 0: none
    slopes: Optional[np.ndarray] = None       # [H]: minus slope times distance
    bias: Optional[np.ndarray] = None         # [H, buckets]: plus bias[h, bucket(distance)]
    buckets: Optional[Sequence[int]] = None   # bucket of distances 0 .. len - 1 (the last: and beyond)
    prefix_lens: Sequence[int] = ()           # tokens of each sample's prefix
    bidirectional: bool = False               # the prefix attends to itself in both directions


#: A bias at or below this (the fp32 number nearest -1e37) hides the key, as minus infinity does.
HIDDEN = float(np.float32(-1e37))


def _sample_scores(q, k, scale, s: Scores, h, prefix):
    """Scores, their tanh (or None), visibility and distances of one head of one sample."""
    m = q.shape[0]
    at = np.arange(m)
    dist = at[:, None] - at[None, :]
    seen = dist >= 0
    if s.bidirectional:
        seen = seen | ((at[:, None] < prefix) & (at[None, :] < prefix))
    x = scale * (q @ k.T)
    t = None
    if s.softcap:
        t = np.tanh(x / s.softcap)
        x = s.softcap * t
    if s.slopes is not None:
        x = x - float(_f64(s.slopes)[h]) * np.abs(dist)
    if s.bias is not None:
        table = _f64(s.bias)[h][np.asarray(s.buckets)]
        far = np.minimum(np.abs(dist), len(s.buckets) - 1)
        b = table[far]
        seen = seen & (b > HIDDEN)
        x = x + np.where(b > HIDDEN, b, 0.0)
    return x, t, seen, dist


def _softmax(x, seen):
    """Probabilities and lse; a row that sees nothing has probabilities 0 and lse -inf."""
    y = np.where(seen, x, -np.inf)
    top = y.max(-1, keepdims=True, initial=-np.inf)
    safe = np.where(np.isfinite(top), top, 0.0)
    e = np.where(seen, np.exp(np.where(seen, x, 0.0) - safe), 0.0)
    total = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, safe + np.log(total), -np.inf)[:, 0]
    return e / np.where(total > 0, total, 1.0), lse


def scored_attention(q, k, v, cu, scale, s: Scores, dout=None):
    """``(out, lse)``, and with dout ``(out, lse, dq, dk, dv, dbias)`` (dbias None
    without a learned bias).  Layouts as the CUDA path: ``[T, heads, d]``, lse ``[H, T]``."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    T, H, _ = q.shape
    G = H // k.shape[1]
    out, lse = np.zeros_like(q), np.zeros((H, T))
    if dout is not None:
        do_all = _f64(dout)
        dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
        dbias = None if s.bias is None else np.zeros(_f64(s.bias).shape)
    for i in range(len(cu) - 1):
        rows = slice(cu[i], cu[i + 1])
        if cu[i + 1] == cu[i]:
            continue
        prefix = s.prefix_lens[i] if len(s.prefix_lens) else 0
        for h in range(H):
            qh, kh, vh = q[rows, h], k[rows, h // G], v[rows, h // G]
            x, t, seen, dist = _sample_scores(qh, kh, scale, s, h, prefix)
            p, lse[h, rows] = _softmax(x, seen)
            out[rows, h] = p @ vh
            if dout is None:
                continue
            do = do_all[rows, h]
            ds = p * (do @ vh.T - (do * out[rows, h]).sum(-1, keepdims=True))
            dv[rows, h // G] += p.T @ do
            if dbias is not None:
                far = np.minimum(np.abs(dist), len(s.buckets) - 1)
                np.add.at(dbias[h], np.asarray(s.buckets)[far].ravel(), ds.ravel())
            if t is not None:
                ds = ds * (1 - t * t)
            dq[rows, h] = scale * (ds @ kh)
            dk[rows, h // G] += scale * (ds.T @ qh)
    if dout is None:
        return out, lse
    return out, lse, dq, dk, dv, dbias
