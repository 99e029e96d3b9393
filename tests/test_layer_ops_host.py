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


def _ffn_desc(**over):
    f = B.GatedFfnDesc()
    f.dtype, f.grad_dtype, f.activation, f.T, f.D, f.F, f.D_out = 1, 1, 0, 4, 64, 128, 32
    f.x_stride, f.w_gate_stride, f.w_up_stride, f.w_down_stride, f.dy_stride = 64, 64, 64, 128, 32
    for k, v in over.items():
        setattr(f, k, v)
    return f


def _ffn_fwd(f, x=A, wg=A, wu=A, wd=A, y=A, gate=A, up=A, ws=A, n=0):
    return B.lib().cp_gated_ffn_fwd(f, x, wg, wu, wd, y, gate, up, ws, n, None)


def _ffn_bwd(f, x=A, wg=A, wu=A, wd=A, gate=A, up=A, dy=A, dx=A, dwg=A, dwu=A, dwd=A, ws=A, n=0):
    return B.lib().cp_gated_ffn_bwd(f, x, wg, wu, wd, gate, up, dy, dx, dwg, dwu, dwd, ws, n, None)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=7), 3), (dict(grad_dtype=5), 3), (dict(dtype=0, grad_dtype=1), 3), (dict(activation=3), 1),
    (dict(activation=-1), 1), (dict(T=-1), 1), (dict(D=0), 2), (dict(D=60), 2), (dict(F=4), 2), (dict(D_out=12), 2),
    (dict(F=(1 << 20) + 8), 2), (dict(x_stride=56), 2), (dict(dy_stride=0), 2), (dict(w_gate_stride=-64), 2),
    (dict(w_down_stride=120), 2), (dict(x_stride=68), 4), (dict(w_up_stride=66), 4), (dict(x_stride=1 << 40), 2)])
def test_gated_ffn_descriptors(cplib, over, status):
    f = _ffn_desc(**over)
    assert _ffn_fwd(f) == status and _ffn_bwd(f) == status
    assert B.lib().cp_last_error()
    assert B.lib().cp_gated_ffn_fwd_workspace_size(f) == 0 and B.lib().cp_gated_ffn_bwd_workspace_size(f) == 0


def test_gated_ffn_pointers(cplib):
    f = _ffn_desc()
    assert _ffn_fwd(None) == 1 and _ffn_bwd(None) == 1
    for name in ("x", "wg", "wu", "wd", "y", "gate", "up"):
        assert _ffn_fwd(f, **{name: None}) == 1, name
        assert _ffn_fwd(f, **{name: A8}) == 4, name
    for name in ("x", "wg", "wu", "wd", "gate", "up", "dy"):
        assert _ffn_bwd(f, **{name: None}) == 1, name
    for name in ("x", "wg", "wu", "wd", "gate", "up", "dy", "dx", "dwg", "dwu", "dwd"):
        assert _ffn_bwd(f, **{name: A8}) == 4, name
    assert _ffn_fwd(f, ws=None) == 5 and _ffn_bwd(f, ws=None) == 5
    # nothing to do
    assert _ffn_fwd(_ffn_desc(T=0), None, None, None, None, None, None, None, None) == 0
    assert _ffn_bwd(_ffn_desc(T=0), dx=None, dwg=None, dwu=None, dwd=None, ws=None) == 0
    assert _ffn_bwd(f, dx=None, dwg=None, dwu=None, dwd=None, ws=None) == 0


def test_rows_that_need_a_copy():
    from vlm_zigzag_head_gb300.ffn import _aligned
    x = torch.zeros(6, 64, dtype=torch.bfloat16)
    assert _aligned(x) is x and _aligned(x[:, :32]).data_ptr() == x.data_ptr()
    for view in (x[:, 1:9], x[:1].expand(6, 64), x.t(), torch.zeros(6, 36, dtype=torch.bfloat16)[:, :32],
                 x[:, :1].expand(6, 64)):
        got = _aligned(view)
        assert got.data_ptr() % 16 == 0 and got.is_contiguous() and torch.equal(got, view)
    assert _aligned(x[2]).data_ptr() == x[2].data_ptr()
