"""Rotation of heads, and its gradient, against the fp64 oracle.

Tolerances, derived from the arithmetic.  With u = 2^-24: cosine and sine are off by 2 steps plus
the angle's own rounding of pi 2^-25 < 2 u, so by under 6 u of 1; the amplitude's product and its
rounding to fp32 add 2 u; the two products and the sum add 3 u: 11 u times amplitude (|x_i| +
|x_j|), so 22 u times amplitude times the row's largest magnitude.  Results in bf16 add half a step
of bf16, 2^-8 of the value.  Elements that are not rotated are equal to the bit."""
import math

import numpy as np
import pytest
import torch

from gpu_util import to64
from oracle import layer as O

DEV = "cuda:0"
U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _heads(T, H, Hkv, d, dtype, layout, g):
    if layout == "fused":       # slices of one projection's output
        qkv = torch.randn((T, H + 2 * Hkv, d), generator=g).to(dtype).to(DEV)
        return qkv[:, :H], qkv[:, H:H + Hkv]
    if layout == "heads":       # [heads][T][d] storage
        q = torch.randn((H, T, d), generator=g).to(dtype).to(DEV).transpose(0, 1)
        k = torch.randn((Hkv, T, d), generator=g).to(dtype).to(DEV).transpose(0, 1)
        return q, k
    if layout == "odd":         # rows that start off the 8-byte grid
        q = torch.randn((T, H, d + 3), generator=g).to(dtype).to(DEV)[..., 1:d + 1]
        k = torch.randn((T, Hkv, d + 3), generator=g).to(dtype).to(DEV)[..., 2:d + 2]
        return q, k
    return (torch.randn((T, h, d), generator=g).to(dtype).to(DEV) for h in (H, Hkv))


def _check(got, x, pos, rot, freqs, sections, inter, amp, sign=1.0):
    want = O.rope(x, pos.cpu(), rot, freqs, sections, inter, amp, sign)
    tol = HALF_STEP[x.dtype] * np.abs(want) + 22 * U * abs(amp) * np.abs(to64(x)).max(-1, keepdims=True)
    err = np.abs(to64(got) - want)
    assert np.all(err <= tol), float((err / tol).max())
    assert torch.equal(got[..., rot:], x[..., rot:])


CASES = [   # T, H, Hkv, d, dtype, layout, rot, sections, interleaved, amplitude
    (1, 32, 8, 128, "bf16", "fused", 128, [64], False, 1.25),
    (1, 1, 1, 64, "f32", "plain", 64, [32], False, 1.0),
    (5, 3, 2, 64, "bf16", "odd", 32, [16], False, 0.5),
    (37, 5, 5, 128, "f32", "heads", 64, [32], True, 1.0),
    (65, 32, 8, 128, "bf16", "fused", 128, [16, 24, 24], False, 1.277),
    (33, 7, 1, 64, "bf16", "heads", 16, [2, 6], True, -1.5),
    (17, 2, 1, 128, "bf16", "odd", 128, [64], True, 1.0),
    (9, 2, 2, 64, "f32", "odd", 64, [8, 8, 8, 8], False, 1.0),
    (21, 6, 3, 128, "bf16", "plain", 0, [0], False, 3.0),
    (1259, 16, 16, 64, "bf16", "fused", 64, [32], False, 1.0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,Hkv,d,dtype,layout,rot,sections,inter,amp", CASES)
def test_matches_oracle(T, H, Hkv, d, dtype, layout, rot, sections, inter, amp):
    import vlm_zigzag_head_gb300 as cp
    g = torch.Generator().manual_seed(T + d)
    q, k = _heads(T, H, Hkv, d, DT[dtype], layout, g)
    axes = len(sections)
    pos = torch.randint(0, 1 << 17, (axes, T) if axes > 1 else (T,), generator=g).to(torch.int32).to(DEV)
    freqs = cp.rope_frequencies(rot, 500000.0, scaling="by_parts", factor=4.0) if rot else ()
    opt = dict(rot_dim=rot, sections=sections, interleaved=inter, inv_freq=freqs, amplitude=amp)
    qo, ko = cp.cp_rope_fwd(q, k, pos, **opt)
    assert qo.is_contiguous() and ko.is_contiguous() and qo.dtype == q.dtype
    _check(qo, q, pos, rot, freqs, sections, inter, amp)
    _check(ko, k, pos, rot, freqs, sections, inter, amp)
    dq, dk = cp.cp_rope_bwd(q, k, pos, **opt)
    _check(dq, q, pos, rot, freqs, sections, inter, amp, -1.0)
    _check(dk, k, pos, rot, freqs, sections, inter, amp, -1.0)
    # in place: the same bits, and nothing beside the heads is touched
    base = q._base if q._base is not None else q
    before = base.clone()
    q0, k0 = q.clone(), k.clone()
    version = q._version
    iq, ik = cp.cp_rope_fwd(q, k, pos, **opt, inplace=True)
    assert iq is q and ik is k and q._version > version
    assert torch.equal(q, qo) and torch.equal(k, ko)
    q.copy_(q0)
    k.copy_(k0)
    assert torch.equal(base, before)


@pytest.mark.gpu
def test_extreme_positions_and_frequencies():
    """Every int32 position has its exact angle (up to the double of a turn count, 2^-49 turns a
    position at 16 turns); defaults are the unscaled frequencies."""
    import vlm_zigzag_head_gb300 as cp
    pos = torch.tensor([0, 1, -1, 131071, 2 ** 31 - 1, -2 ** 31, 99999999], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(3)
    q, k = _heads(7, 2, 1, 64, torch.float32, "plain", g)
    freqs = [1.0, -0.25, 7.5, 0.0, 3.14159, 1e-9, 2 * np.pi, 100.25] * 4
    qo, _ = cp.cp_rope_fwd(q, k, pos, inv_freq=freqs)
    want = O.rope(q, pos.cpu(), 64, freqs, [32], False)
    far = np.abs(to64(pos))[:, None, None] * 2 * np.pi * 2.0 ** -49
    assert np.all(np.abs(to64(qo) - want) <= (23 * U + 2 * far) * np.abs(to64(q)).max(-1, keepdims=True))
    qo, _ = cp.cp_rope_fwd(q, k, pos[:4].repeat(2)[:7].contiguous())
    _check(qo, q, pos[:4].repeat(2)[:7], 64, [10000.0 ** (-p / 32) for p in range(32)], [32], False, 1.0)


@pytest.mark.gpu
def test_nonfinite_stays_in_its_pair_and_no_tokens():
    import vlm_zigzag_head_gb300 as cp
    g = torch.Generator().manual_seed(4)
    q, k = _heads(6, 2, 1, 64, torch.bfloat16, "plain", g)
    pos = torch.arange(6, dtype=torch.int32, device=DEV)
    clean = cp.cp_rope_fwd(q, k, pos, rot_dim=32)[0]
    bad = q.clone()
    bad[2, 1, 3], bad[4, 0, 40] = float("nan"), float("inf")
    got = cp.cp_rope_fwd(bad, k, pos, rot_dim=32)[0]
    touched = torch.zeros_like(got, dtype=torch.bool)
    touched[2, 1, 3] = touched[2, 1, 19] = touched[4, 0, 40] = True
    assert torch.equal(got[~touched], clean[~touched])
    assert got[2, 1, 3].isnan() and got[2, 1, 19].isnan() and got[4, 0, 40] == float("inf")
    e = cp.cp_rope_fwd(q[:0], k[:0], pos[:0])
    assert e[0].shape == (0, 2, 64) and e[1].shape == (0, 1, 64)


@pytest.mark.gpu
def test_autograd_streams_and_graphs():
    import vlm_zigzag_head_gb300 as cp
    from vlm_zigzag_head_gb300.autograd import rope
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn((50, 8, 64), generator=g).to(DEV).requires_grad_(True)
    pos = torch.arange(50, dtype=torch.int32, device=DEV) + 1000
    opt = dict(rot_dim=48, interleaved=True, amplitude=1.1)
    q, k = rope(qkv[:, :4], qkv[:, 4:6], pos, **opt)
    dq, dk = torch.randn(q.shape, generator=g).to(DEV), torch.randn(k.shape, generator=g).to(DEV)
    d, = torch.autograd.grad((q, k), qkv, (dq, dk))
    freqs = [10000.0 ** (-p / 24) for p in range(24)]
    _check(d[:, :4].contiguous(), dq, pos, 48, freqs, [24], True, 1.1, -1.0)
    _check(d[:, 4:6].contiguous(), dk, pos, 48, freqs, [24], True, 1.1, -1.0)
    assert not d[:, 6:].any()
    # only one output used, and a gradient whose last dimension is not contiguous
    q, k = rope(qkv[:, :4], qkv[:, 4:6], pos, **opt)
    d1, = torch.autograd.grad(k, qkv, dk.transpose(0, 2).contiguous().transpose(0, 2))
    assert torch.equal(d1[:, 4:6], d[:, 4:6]) and not d1[:, :4].any()
    # the map is linear: <R x, y> = <x, R^T y> against the forward
    lhs = (to64(q) * to64(dq)).sum() + (to64(k) * to64(dk)).sum()
    rhs = (to64(qkv) * to64(d)).sum()
    assert abs(lhs - rhs) <= 1e-5 * (np.abs(to64(q) * to64(dq)).sum() + np.abs(to64(k) * to64(dk)).sum())
    x = qkv.detach()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qs, ks = cp.cp_rope_fwd(x[:, :4], x[:, 4:6], pos, **opt)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(qs, q) and torch.equal(ks, k)
    graph = torch.cuda.CUDAGraph()
    work = x.clone()
    with torch.cuda.graph(graph):
        cp.cp_rope_fwd(work[:, :4], work[:, 4:6], pos, **opt, inplace=True)
    work.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(work[:, :4], q) and torch.equal(work[:, 4:6], k) and torch.equal(work[:, 6:], x[:, 6:])


def test_frequencies():
    import vlm_zigzag_head_gb300 as cp
    base = [10000.0 ** (-2 * p / 64) for p in range(32)]
    assert np.allclose(cp.rope_frequencies(64), base, rtol=1e-15)
    assert np.allclose(cp.rope_frequencies(64, scaling="linear", factor=4.0), np.array(base) / 4, rtol=1e-15)
    b = cp.rope_frequencies(64, scaling="base", factor=4.0)
    assert b[0] == 1.0 and math.isclose(b[-1], base[-1] / 4, rel_tol=1e-12)
    p = cp.rope_frequencies(64, scaling="by_parts", factor=8.0, trained_length=4096, low=1.0, high=4.0)
    turns = np.array(base) * 4096 / (2 * math.pi)
    assert np.allclose(np.array(p)[turns >= 4], np.array(base)[turns >= 4], rtol=1e-15)
    assert np.allclose(np.array(p)[turns <= 1], np.array(base)[turns <= 1] / 8, rtol=1e-15)
    assert all(f / 8 <= v <= f * (1 + 1e-12) for f, v in zip(base, p))
    assert cp.rope_frequencies(0) == ()
    from vlm_zigzag_head_gb300 import rope
    odd = (np.float32(1.0), 2, np.float64(0.5)) + (0.25,) * 29      # entries of any kind of number
    f = rope._desc(1, (1, 1, 64), (64, 64, 1), (1, 1, 64), (64, 64, 1), (1,), 1e4, None, None, False,
                   rope.Frequencies(float(x) for x in odd), 1.0, False)
    assert [f.inv_freq[i] for i in range(4)] == [1.0, 2.0, 0.5, 0.25]
    for bad in (dict(rot_dim=7), dict(rot_dim=64, scaling="cubic"), dict(rot_dim=64, factor=0.0),
                dict(rot_dim=64, theta=-1.0), dict(rot_dim=2, scaling="base", factor=2.0),
                dict(rot_dim=64, scaling="by_parts", low=2.0, high=2.0)):
        with pytest.raises(cp.CpError):
            cp.rope_frequencies(**bad)
