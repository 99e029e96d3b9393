"""Query / key norm with rotation against the fp64 oracle.

Tolerances, derived from the arithmetic.  With u = 2^-24 (half a step of fp32): the sum of squares
is off by at most 12 u (8 fused adds and 4 shuffle adds), its root by half of that plus 2 u for the
reciprocal root; the two products of z add 2 u; cosine and sine are off by 2 steps plus the angle's
own rounding of pi 2^-25 < 2 u; the rotation adds 2 u.  Together under 16 u times |z_i| + |z_j|, so
32 u times the row's largest |z|.  The backward repeats these steps twice more: 96 u times r times
the largest |g w| (1 + largest |n|).  A weight gradient sums at most 200 terms a lane here, then at
most 60 more partial sums: 256 u times the sum of magnitudes.  Results in bf16 add half a step of
bf16, 2^-8 of the value."""
import numpy as np
import pytest
import torch

from gpu_util import to64
from oracle import scored as O

DEV = "cuda:0"
U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _freqs(rot, theta=10000.0):
    return [theta ** (-2.0 * p / rot) for p in range(rot // 2)]


def _inputs(T, H, Hkv, d, dtype, layout, seed, axes=1, pos=None):
    g = torch.Generator().manual_seed(seed)
    if layout == "fused":       # slices of one projection's output
        qkv = torch.randn((T, H + 2 * Hkv, d), generator=g).to(dtype).to(DEV)
        q, k = qkv[:, :H], qkv[:, H:H + Hkv]
    elif layout == "heads":     # [heads][T][d] storage
        q = torch.randn((H, T, d), generator=g).to(dtype).to(DEV).transpose(0, 1)
        k = torch.randn((Hkv, T, d), generator=g).to(dtype).to(DEV).transpose(0, 1)
    elif layout == "odd":       # rows that start off the 16-byte grid
        q = torch.randn((T, H, d + 3), generator=g).to(dtype).to(DEV)[..., 1:d + 1]
        k = torch.randn((T, Hkv, d + 3), generator=g).to(dtype).to(DEV)[..., 2:d + 2]
    else:
        q = torch.randn((T, H, d), generator=g).to(dtype).to(DEV)
        k = torch.randn((T, Hkv, d), generator=g).to(dtype).to(DEV)
    if pos is None:
        pos = torch.randint(0, 1 << 17, (axes, T) if axes > 1 else (T,), generator=g)
    qw, kw = 1 + 0.3 * torch.randn(d, generator=g), 1 + 0.3 * torch.randn(d, generator=g)
    dq, dk = torch.randn((T, H, d), generator=g).to(dtype), torch.randn((T, Hkv, d), generator=g).to(dtype)
    return q, k, pos.to(torch.int32).to(DEV), qw.to(DEV), kw.to(DEV), dq.to(DEV), dk.to(DEV)


def _check_fwd(got, x, pos, w, eps, rot, freqs, sections, inter):
    assert got.dtype == x.dtype and got.is_contiguous()
    want = O.norm_rope_fwd(x, pos.cpu(), w, eps, rot, freqs, sections, inter)
    z = O.norm_rope_fwd(x, pos.cpu(), w, eps, 0, [], [0] * len(sections), inter)
    err = np.abs(to64(got) - want)
    tol = HALF_STEP[x.dtype] * np.abs(want) + 32 * U * np.abs(z).max(-1, keepdims=True)
    assert np.all(err <= tol), float((err / tol).max())


def _check_bwd(dx, dw, x, dy, pos, w, eps, rot, freqs, sections, inter):
    wdx, wdw = O.norm_rope_bwd(x, dy, pos.cpu(), w, eps, rot, freqs, sections, inter)
    x64, w64 = to64(x), np.ones(x.shape[-1]) if w is None else to64(w)
    r = 1 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + eps)
    i, j, ang = O.rope_matrix_parts(pos.cpu(), rot, freqs, sections, inter)
    g = O._rotate(to64(dy), i, j, ang, -1.0)
    big = np.abs(to64(dy)).max(-1, keepdims=True) * 1.5 * np.abs(w64).max()
    tol = HALF_STEP[x.dtype] * np.abs(wdx) + 96 * U * r * big * (1 + np.abs(x64 * r).max(-1, keepdims=True))
    err = np.abs(to64(dx) - wdx)
    assert np.all(err <= tol), float((err / tol).max())
    if w is not None:
        tol = 256 * U * np.abs(g * x64 * r).sum((0, 1))
        err = np.abs(to64(dw) - wdw)
        assert np.all(err <= tol), float((err / tol).max())


CASES = [   # T, H, Hkv, d, dtype, layout, rot, sections, interleaved
    (1, 4, 1, 128, "bf16", "plain", 128, [64], False),
    (1, 1, 1, 64, "f32", "fused", 64, [32], False),
    (5, 3, 2, 64, "bf16", "odd", 32, [16], False),
    (37, 5, 5, 128, "f32", "heads", 64, [32], True),
    (65, 32, 8, 128, "bf16", "fused", 128, [16, 24, 24], False),
    (33, 7, 1, 64, "bf16", "heads", 16, [2, 6], True),
    (17, 2, 1, 128, "bf16", "odd", 128, [64], True),
    (9, 2, 2, 64, "f32", "odd", 64, [8, 8, 8, 8], False),
    (21, 6, 3, 128, "bf16", "plain", 0, [0], False),
    (259, 16, 16, 64, "bf16", "fused", 64, [32], False),
]
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,Hkv,d,dtype,layout,rot,sections,inter", CASES)
def test_forward_and_backward_match_oracle(T, H, Hkv, d, dtype, layout, rot, sections, inter):
    from vlm_zigzag_head_gb300 import cp_qk_norm_rope_bwd, cp_qk_norm_rope_fwd
    q, k, pos, qw, kw, dqo, dko = _inputs(T, H, Hkv, d, DT[dtype], layout, T + d, len(sections))
    opt = dict(eps=1e-6, rot_dim=rot, sections=sections, interleaved=inter)
    tail = (1e-6, rot, _freqs(rot) if rot else [], sections, inter)
    qo, ko = cp_qk_norm_rope_fwd(q, k, pos, qw, kw, **opt)
    _check_fwd(qo, q, pos, qw, *tail)
    _check_fwd(ko, k, pos, kw, *tail)
    dq, dk, dqw, dkw = cp_qk_norm_rope_bwd(q, k, pos, dqo, dko, qw, kw, **opt)
    _check_bwd(dq, dqw, q, dqo, pos, qw, *tail)
    _check_bwd(dk, dkw, k, dko, pos, kw, *tail)
    # the same call again gives the same bits: the sums do not depend on timing
    again = cp_qk_norm_rope_bwd(q, k, pos, dqo, dko, qw, kw, **opt)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dqw, dkw), again))


@pytest.mark.gpu
def test_extreme_positions_and_custom_frequencies():
    """Every int32 position has its exact angle; frequencies of any sign and size."""
    from vlm_zigzag_head_gb300 import cp_qk_norm_rope_fwd
    pos = torch.tensor([0, 1, -1, 131071, 2 ** 31 - 1, -2 ** 31, 99999999], dtype=torch.int32)
    q, k, pos, qw, kw, _, _ = _inputs(7, 2, 1, 64, torch.float32, "plain", 3, pos=pos)
    freqs = [1.0, -0.25, 7.5, 0.0, 3.14159, 1e-9, 2 * np.pi, 100.25] * 4
    qo, ko = cp_qk_norm_rope_fwd(q, k, pos, qw, kw, inv_freq=freqs, eps=0.0)
    _check_far(qo, q, pos, qw, freqs)
    _check_far(ko, k, pos, kw, freqs)


def _check_far(got, x, pos, w, freqs):
    """The turns per position are doubles: a position of 2^31 times half a step of a turn count of
    16 is 2^31 2^-49 = 4e-6 turns, so the tolerance grows with the position (2 pi 2^-49 each)."""
    want = O.norm_rope_fwd(x, pos.cpu(), w, 0.0, 64, freqs, [32], False)
    z = O.norm_rope_fwd(x, pos.cpu(), w, 0.0, 0, [], [0], False)
    far = np.abs(to64(pos))[:, None, None] * 2 * np.pi * 2.0 ** -49
    err = np.abs(to64(got) - want)
    assert np.all(err <= (34 * U + 2 * far) * np.abs(z).max(-1, keepdims=True))


@pytest.mark.gpu
def test_weights_in_bf16_missing_and_no_tokens():
    from vlm_zigzag_head_gb300 import cp_qk_norm_rope_bwd, cp_qk_norm_rope_fwd
    q, k, pos, qw, kw, dqo, dko = _inputs(11, 4, 2, 128, torch.bfloat16, "plain", 5)
    tail = (1e-5, 128, _freqs(128), [64], False)
    qw16 = qw.to(torch.bfloat16)
    qo, ko = cp_qk_norm_rope_fwd(q, k, pos, qw16, None, eps=1e-5)
    _check_fwd(qo, q, pos, qw16, *tail)
    _check_fwd(ko, k, pos, None, *tail)
    dq, dk, dqw, dkw = cp_qk_norm_rope_bwd(q, k, pos, dqo, dko, qw16, None, eps=1e-5)
    assert dkw is None and dqw.dtype == torch.float32
    _check_bwd(dq, dqw, q, dqo, pos, qw16, *tail)
    _check_bwd(dk, None, k, dko, pos, None, *tail)
    e = q[:0], k[:0], pos[:0]
    qo, ko = cp_qk_norm_rope_fwd(*e, qw, kw)
    assert qo.shape == (0, 4, 128) and ko.shape == (0, 2, 128)
    _, _, dqw, dkw = cp_qk_norm_rope_bwd(*e, dqo[:0], dko[:0], qw, kw)
    assert not dqw.any() and not dkw.any()


@pytest.mark.gpu
def test_zero_rows_large_values_and_nan_stay_in_their_row():
    """eps keeps an all-zero row at zero; a NaN or infinity reaches its own row alone."""
    from vlm_zigzag_head_gb300 import cp_qk_norm_rope_bwd, cp_qk_norm_rope_fwd
    q, k, pos, qw, kw, dqo, dko = _inputs(6, 3, 3, 64, torch.bfloat16, "plain", 9)
    q[0, 1] = 0
    q[2, 0, 5] = float("nan")
    k[4, 2, 3] = float("inf")
    q[3] *= 1e15
    qo, ko = cp_qk_norm_rope_fwd(q, k, pos, qw, kw)
    assert not qo[0, 1].any()
    bad = ~torch.isfinite(qo).all(-1)
    assert bad.nonzero().tolist() == [[2, 0]]
    assert (~torch.isfinite(ko).all(-1)).nonzero().tolist() == [[4, 2]]
    dq, dk, _, _ = cp_qk_norm_rope_bwd(q, k, pos, dqo, dko, qw, kw)
    assert (~torch.isfinite(dq).all(-1)).nonzero().tolist() == [[2, 0]]
    assert (~torch.isfinite(dk).all(-1)).nonzero().tolist() == [[4, 2]]


@pytest.mark.gpu
def test_weight_gradient_without_eps_ignores_idle_lanes():
    """eps = 0 and an odd head count: the lanes past the last head add nothing."""
    from vlm_zigzag_head_gb300 import cp_qk_norm_rope_bwd
    q, k, pos, qw, kw, dqo, dko = _inputs(13, 1, 2, 64, torch.float32, "plain", 21)
    dq, dk, dqw, dkw = cp_qk_norm_rope_bwd(q, k, pos, dqo, dko, qw, kw, eps=0.0)
    tail = (0.0, 64, _freqs(64), [32], False)
    _check_bwd(dq, dqw, q, dqo, pos, qw, *tail)
    _check_bwd(dk, dkw, k, dko, pos, kw, *tail)


@pytest.mark.gpu
def test_autograd_and_strided_gradients():
    from vlm_zigzag_head_gb300.autograd import qk_norm_rope
    q, k, pos, qw, kw, dqo, dko = _inputs(19, 4, 2, 64, torch.bfloat16, "fused", 2)
    leaves = [t.detach().clone().requires_grad_(True) for t in (q, k, qw, kw)]
    qo, ko = qk_norm_rope(leaves[0], leaves[1], pos, leaves[2], leaves[3], rot_dim=32)
    # gradients that arrive with other strides
    gq = dqo.transpose(0, 1).contiguous().transpose(0, 1)
    got = torch.autograd.grad((qo, ko), leaves, (gq, dko))
    tail = (1e-6, 32, _freqs(32), [16], False)
    _check_bwd(got[0], got[2], q, dqo, pos, qw, *tail)
    _check_bwd(got[1], got[3], k, dko, pos, kw, *tail)
    # one output unused, one leaf without a gradient
    qo, ko = qk_norm_rope(leaves[0], k, pos, leaves[2], kw, rot_dim=32)
    dq, dqw = torch.autograd.grad(qo, (leaves[0], leaves[2]), dqo)
    assert torch.equal(dq, got[0]) and torch.equal(dqw, got[2])


@pytest.mark.gpu
def test_graph_replay_and_side_stream():
    """Captured forward and backward replay on new values; a side stream gives the same bits."""
    from vlm_zigzag_head_gb300 import cp_qk_norm_rope_bwd, cp_qk_norm_rope_fwd
    args = _inputs(70, 8, 2, 128, torch.bfloat16, "plain", 31)
    q, k, pos, qw, kw, dqo, dko = args

    def both():
        return cp_qk_norm_rope_fwd(q, k, pos, qw, kw) + cp_qk_norm_rope_bwd(q, k, pos, dqo, dko, qw, kw)
    want0 = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want0))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = both()
    q.mul_(2).add_(1)
    dko.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, both()))


@pytest.mark.gpu
def test_python_refusals_on_device():
    from vlm_zigzag_head_gb300 import CpError, cp_qk_norm_rope_bwd, cp_qk_norm_rope_fwd
    q, k, pos, qw, kw, dqo, dko = _inputs(4, 2, 1, 64, torch.bfloat16, "plain", 1)
    bad = [lambda: cp_qk_norm_rope_fwd(q.half(), k.half(), pos), lambda: cp_qk_norm_rope_fwd(q, k.float(), pos),
           lambda: cp_qk_norm_rope_fwd(q, k[:3], pos), lambda: cp_qk_norm_rope_fwd(q, k, pos.long()),
           lambda: cp_qk_norm_rope_fwd(q, k, pos[:3]), lambda: cp_qk_norm_rope_fwd(q, k, pos.cpu()),
           lambda: cp_qk_norm_rope_fwd(q[..., ::2], k[..., ::2], pos), lambda: cp_qk_norm_rope_fwd(q, k, pos, qw[:3]),
           lambda: cp_qk_norm_rope_fwd(q, k, pos, qw, kw.to(torch.bfloat16)),
           lambda: cp_qk_norm_rope_fwd(q, k, pos, rot_dim=8), lambda: cp_qk_norm_rope_fwd(q, k, pos, theta=-1.0),
           lambda: cp_qk_norm_rope_fwd(q, k, pos.expand(3, 4).contiguous()),
           lambda: cp_qk_norm_rope_fwd(q, k, pos, inv_freq=[1.0]),
           lambda: cp_qk_norm_rope_fwd(q, k, pos, sections=[16, 16]),
           lambda: cp_qk_norm_rope_bwd(q, k, pos, dqo.float(), dko),
           lambda: cp_qk_norm_rope_bwd(q, k, pos, dqo[:2], dko)]
    for i, call in enumerate(bad):
        with pytest.raises(CpError):
            call()
            pytest.fail("call %d was not refused" % i)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["fused", "heads", "odd"])
def test_saved_tensors_that_come_back_with_other_strides(layout):
    """Offloading keeps contiguous copies of the strided q and k: the backward reads those."""
    from vlm_zigzag_head_gb300.autograd import qk_norm_rope
    q, k, pos, qw, kw, dqo, dko = _inputs(19, 4, 2, 64, torch.bfloat16, layout, 2, axes=2)
    leaves = [t.detach().requires_grad_(True) for t in (q, k, qw, kw)]
    sections = [20, 12]

    def run():
        qo, ko = qk_norm_rope(leaves[0], leaves[1], pos, leaves[2], leaves[3], sections=sections)
        return qo, ko
    want = torch.autograd.grad(run(), leaves, (dqo, dko))
    with torch.autograd.graph.save_on_cpu():
        outs = run()
    sections.clear()   # the options are those of the forward
    got = torch.autograd.grad(outs, leaves, (dqo, dko))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_offsets_past_32_bits(dtype):
    """The last rows of tensors with more than 2^31 elements get the bits that they get alone."""
    from vlm_zigzag_head_gb300 import cp_qk_norm_rope_bwd, cp_qk_norm_rope_fwd
    H, d, n = 64, 64, 70
    T = 2 ** 31 // (H * d) + n
    x = torch.zeros((T, H + 1, d), dtype=dtype, device=DEV)
    tail = torch.randn((n, H + 1, d), device=DEV, generator=torch.Generator(DEV).manual_seed(3)).to(dtype)
    x[-n:] = tail
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    w = torch.linspace(0.5, 1.5, d, device=DEV)
    ends = []
    for y, p in ((x, pos), (tail, pos[-n:].contiguous())):
        q, k = y[:, :H], y[:, H:]
        qo, ko = cp_qk_norm_rope_fwd(q, k, p, w, w)
        dq, dk, dw, _ = cp_qk_norm_rope_bwd(q, k, p, qo, ko, w, w)
        ends.append([t[-n:].clone() for t in (qo, ko, dq, dk)])
        assert torch.isfinite(dw).all()
    assert all(torch.equal(a, b) for a, b in zip(*ends))
    del x, y, q, k, qo, ko, dq, dk
    torch.cuda.empty_cache()
