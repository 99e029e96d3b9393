"""Refusals of the query / key norm with rotation: every bad argument gives its documented status
before anything is launched (no GPU)."""
import ctypes

import pytest
import torch

from vlm_zigzag_head_gb300 import CpError, _binding as B, cp_qk_norm_rope_fwd


def _desc(**over):
    f = B.NormRopeDesc()
    f.dtype, f.weight_dtype, f.T, f.H, f.H_kv, f.d = 1, 0, 4, 2, 1, 64
    f.q_stride_t, f.q_stride_h, f.k_stride_t, f.k_stride_h = 128, 64, 64, 64
    f.rot_dim, f.interleaved, f.n_axes, f.eps = 64, 0, 1, 1e-6
    f.sections[0] = 32
    f.inv_freq = (ctypes.c_double * 32)(*([1.0] * 32))
    for k, v in over.items():
        if k == "sections":
            for i, n in enumerate(v):
                f.sections[i] = n
        else:
            setattr(f, k, v)
    return f


# stand-ins for device pointers: refused calls never touch them
A16, A8 = ctypes.c_void_p(4096), ctypes.c_void_p(4104)


def _fwd(f, q=A16, k=A16, pos=A16, qw=None, kw=None, qo=A16, ko=A16):
    return B.lib().cp_qk_norm_rope_fwd(ctypes.byref(f), q, k, pos, qw, kw, qo, ko, None)


BAD = [(dict(dtype=7), 3), (dict(weight_dtype=9), 3), (dict(T=-1), 1), (dict(H=0), 1), (dict(H_kv=0), 1),
       (dict(H=1 << 21), 2), (dict(d=96), 2), (dict(rot_dim=24), 2), (dict(rot_dim=80), 2), (dict(rot_dim=-16), 2),
       (dict(n_axes=0), 2), (dict(n_axes=5), 2), (dict(sections=[31]), 2), (dict(n_axes=2, sections=[40, -8]), 2),
       (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(inv_freq=None), 1),
       (dict(inv_freq=(ctypes.c_double * 32)(*([1.0] * 31 + [float("nan")]))), 1)]


@pytest.mark.parametrize("over,status", BAD)
def test_bad_descriptors(cplib, over, status):
    assert _fwd(_desc(**over)) == status
    assert B.lib().cp_last_error()


def test_bad_pointers(cplib):
    f = _desc()
    odd = ctypes.c_void_p(4097)
    for name in ("q", "k", "pos", "qo", "ko"):
        assert _fwd(f, **{name: None}) == 1, name
        assert _fwd(f, **{name: odd}) == 4, name
    for name in ("qo", "ko"):       # outputs are written 16 bytes at a time
        assert _fwd(f, **{name: A8}) == 4, name
    assert _fwd(f, qw=ctypes.c_void_p(4098)) == 4
    bwd = B.lib().cp_qk_norm_rope_bwd
    ok = [A16] * 5
    assert bwd(ctypes.byref(f), *ok, A16, A16, A16, None, None, None, None, 0, None) == 1
    assert bwd(ctypes.byref(f), *ok, A8, A16, A16, A16, None, None, None, 0, None) == 4
    assert bwd(ctypes.byref(f), *ok, A16, A16, A16, A16, A16, None, None, 0, None) == 5
    assert bwd(ctypes.byref(f), *ok, A16, A16, A16, A16, A16, None, A8, 0, None) == 4
    assert B.lib().cp_qk_norm_rope_fwd(None, A16, A16, A16, None, None, A16, A16, None) == 1


def test_no_tokens_is_a_no_op(cplib):
    assert _fwd(_desc(T=0), q=None, k=None, pos=None, qo=None, ko=None) == 0


def test_python_refusals():
    x = torch.zeros(4, 2, 64)
    with pytest.raises(CpError):
        cp_qk_norm_rope_fwd(x, x, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(CpError):
        cp_qk_norm_rope_fwd(x[0], x, torch.zeros(4, dtype=torch.int32))


@pytest.mark.parametrize("pos_shape", [(), (3,), (1, 4, 1), (0, 4), (5, 4)])
def test_position_shapes(pos_shape):
    from vlm_zigzag_head_gb300 import norm_rope
    with pytest.raises(CpError):
        norm_rope._desc(1, (4, 2, 64), (128, 64, 1), (4, 1, 64), (64, 64, 1), pos_shape, 0, 1e-6, 1e4, None, None,
                        False, None)
