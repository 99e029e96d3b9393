"""Refusals of the layer norm, the rotation of heads and the gated feed-forward block: every bad
argument gives its documented status before anything is launched (no GPU)."""
import ctypes

import pytest
import torch

from vlm_zigzag_head_gb300 import CpError, _binding as B, cp_layer_norm_fwd, cp_rope_fwd, rope

# stand-ins for device pointers: refused calls never touch them
A, A8, A2, ODD = (ctypes.c_void_p(p) for p in (4096, 4104, 4098, 4097))


def _norm_desc(**over):
    f = B.LayerNormDesc()
    f.dtype, f.weight_dtype, f.T, f.D, f.x_stride, f.dy_stride, f.eps = 1, 0, 4, 64, 64, 64, 1e-5
    for k, v in over.items():
        setattr(f, k, v)
    return f


def _norm_fwd(f, x=A, w=A, b=A, y=A, mean=A, rstd=A):
    return B.lib().cp_layer_norm_fwd(f, x, w, b, y, mean, rstd, None)


def _norm_bwd(f, x=A, dy=A, w=A, mean=A, rstd=A, dx=A, dw=A, db=A, ws=A, n=0):
    return B.lib().cp_layer_norm_bwd(f, x, dy, w, mean, rstd, dx, dw, db, ws, n, None)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=7), 3), (dict(weight_dtype=9), 3), (dict(T=-1), 1), (dict(D=0), 2), (dict(D=16385), 2),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1)])
def test_layer_norm_descriptors(cplib, over, status):
    assert _norm_fwd(_norm_desc(**over)) == status
    assert _norm_bwd(_norm_desc(**over)) == status
    assert B.lib().cp_last_error()
    assert B.lib().cp_layer_norm_bwd_workspace_size(_norm_desc(**over)) == 0


def test_layer_norm_pointers(cplib):
    f = _norm_desc()
    assert _norm_fwd(None) == 1
    for name in ("x", "y"):
        assert _norm_fwd(f, **{name: None}) == 1
    for name in ("x", "w", "b", "y", "mean", "rstd"):
        assert _norm_fwd(f, **{name: ODD}) == 4, name
    assert _norm_fwd(f, y=A8) == 4
    for name in ("x", "dy", "mean", "rstd"):
        assert _norm_bwd(f, **{name: None}) == 1
    for name in ("x", "dy", "w", "mean", "rstd", "dx", "dw", "db"):
        assert _norm_bwd(f, **{name: ODD}) == 4, name
    assert _norm_bwd(f, dx=A8) == 4 and _norm_bwd(f, ws=A8) == 4 and _norm_bwd(f, ws=None) == 5


def test_layer_norm_with_nothing_to_do(cplib):
    assert _norm_fwd(_norm_desc(T=0), x=None, y=None) == 0
    assert _norm_bwd(_norm_desc(T=0), x=None, dy=None, dx=None, dw=None, db=None) == 0
    assert _norm_bwd(_norm_desc(), dx=None, dw=None, db=None, ws=None) == 0


def _rope_desc(**over):
    f = B.RopeDesc()
    f.dtype, f.T, f.H, f.H_kv, f.d = 1, 4, 2, 1, 64
    f.q_stride_t, f.q_stride_h, f.k_stride_t, f.k_stride_h = 128, 64, 64, 64
    f.q_out_stride_t, f.q_out_stride_h, f.k_out_stride_t, f.k_out_stride_h = 128, 64, 64, 64
    f.rot_dim, f.interleaved, f.n_axes, f.amplitude = 64, 0, 1, 1.0
    f.sections[0] = 32
    f.inv_freq = (ctypes.c_double * 32)(*([1.0] * 32))
    for k, v in over.items():
        if k == "sections":
            for i, n in enumerate(v):
                f.sections[i] = n
        else:
            setattr(f, k, v)
    return f


BQ, BK = ctypes.c_void_p(8192), ctypes.c_void_p(16384)


def _rotate(f, q=A, k=A, pos=A, qo=BQ, ko=BK):
    a, b = (fn(f, q, k, pos, qo, ko, None) for fn in (B.lib().cp_rope_fwd, B.lib().cp_rope_bwd))
    assert a == b
    return a


@pytest.mark.parametrize("over,status", [
    (dict(dtype=7), 3), (dict(T=-1), 1), (dict(H=0), 1), (dict(H_kv=0), 1), (dict(H=1 << 21), 2), (dict(d=96), 2),
    (dict(rot_dim=24), 2), (dict(rot_dim=80), 2), (dict(rot_dim=-16), 2), (dict(n_axes=0), 2), (dict(n_axes=5), 2),
    (dict(sections=[31]), 2), (dict(n_axes=2, sections=[40, -8]), 2), (dict(amplitude=float("nan")), 1),
    (dict(amplitude=float("inf")), 1), (dict(inv_freq=None), 1), (dict(q_out_stride_t=0), 1),
    (dict(q_out_stride_h=0), 1), (dict(k_out_stride_t=0), 1),
    (dict(inv_freq=(ctypes.c_double * 32)(*([1.0] * 31 + [float("nan")]))), 1)])
def test_rope_descriptors(cplib, over, status):
    assert _rotate(_rope_desc(**over)) == status
    assert B.lib().cp_last_error()


def test_rope_pointers(cplib):
    f = _rope_desc()
    assert _rotate(None) == 1
    for name in ("q", "k", "pos", "qo", "ko"):
        assert _rotate(f, **{name: None}) == 1, name
        assert _rotate(f, **{name: ODD}) == 4, name
    assert _rotate(_rope_desc(q_stride_t=256), qo=A) == 1      # in place with other strides
    assert _rotate(_rope_desc(T=0), None, None, None, None, None) == 0


def test_python_refusals(cplib):
    x = torch.zeros(4, 2, 64)
    pos = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: cp_layer_norm_fwd(x), lambda: cp_layer_norm_fwd(torch.zeros(())),
                 lambda: cp_rope_fwd(x, x, pos), lambda: cp_rope_fwd(x[0], x, pos)):
        with pytest.raises(CpError):
            call()


def test_heads_that_share_memory_are_seen():
    """What an in-place rotation refuses: heads or tensors that overlap."""
    x = torch.zeros(6, 8, 64)
    assert rope._rows_apart(x.stride(), x.shape) and rope._rows_apart(x.transpose(0, 1).stride(), (8, 6, 64))
    assert not rope._rows_apart(x[:, :1].expand(6, 3, 64).stride(), (6, 3, 64))
    assert not rope._rows_apart(x[:1].expand(6, 8, 64).stride(), (6, 8, 64))
    assert not rope._rows_apart((32, 64, 1), (6, 2, 64))
    assert rope._rows_apart((0, 64, 1), (1, 2, 64))
    assert rope._disjoint(x[:, :4], x[:, 4:6]) and rope._disjoint(x[:, 4:], x[:, :4])
    assert rope._disjoint(x[:3], x[3:])
    t = torch.zeros(8, 6, 64).transpose(0, 1)
    assert rope._disjoint(t[:, :4], t[:, 4:])
    assert not rope._disjoint(x[:, :4], x[:, 3:6]) and not rope._disjoint(x, x)
    assert not rope._disjoint(x[:, ::2], x[:, 1::2])   # apart, but not seen to be: refused
    assert rope._disjoint(x[:1, :4], x[:1, 4:6])
