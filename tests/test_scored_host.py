"""Attention with modified scores without a GPU: plans cover exactly the visible pairs, buckets, and
the refusals of every entry point."""
import ctypes

import numpy as np
import pytest
import torch

from vlm_zigzag_head_gb300 import CpError, _binding as B, relative_buckets
from vlm_zigzag_head_gb300.scored import build_plan


def _host(plan):
    return (ctypes.c_char * len(plan)).from_buffer(plan)


def _pairs(plan):
    n = [ctypes.c_int64() for _ in range(3)]
    B.check(B.lib().cp_score_plan_pairs(_host(plan), *(ctypes.byref(x) for x in n)))
    return [x.value for x in n]


@pytest.mark.parametrize("lens,prefix", [([1], 0), ([257, 0, 1, 640], 0), ([300, 129], 128), ([300, 129], 129),
                                         ([1000, 40], [999, 0]), ([4096], 1), ([128, 128], [128, 64])])
@pytest.mark.parametrize("both", [False, True])
def test_plans_cover_the_visible_pairs(cplib, lens, prefix, both):
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    plan, T = build_plan(cu, 3, prefix, both, None, 152)
    pre = [prefix] * len(lens) if isinstance(prefix, int) else prefix
    want = sum(n * (n + 1) // 2 + (p * (p - 1) // 2 if both else 0) for n, p in zip(lens, pre))
    assert T == sum(lens) and _pairs(plan) == [want] * 3


def test_relative_buckets():
    b = relative_buckets(8, 64)
    assert len(b) == 65 and b[:5] == [0, 1, 2, 3, 4] and b[64] == 7
    # from 4 on the bucket rises at 4 * 2, 4 * 4, 4 * 8: exact powers
    assert [b.index(x) for x in (5, 6, 7)] == [8, 16, 32]
    assert b == sorted(b)
    for bad in ((1, 10), (32, 16)):
        with pytest.raises(CpError):
            relative_buckets(*bad)


@pytest.mark.parametrize("kw", [dict(cu=[0]), dict(cu=[1, 5]), dict(cu=[0, 5, 3]), dict(heads=0), dict(prefix=6),
                                dict(prefix=-1), dict(prefix=[1, 2]), dict(buckets=[0, -1]),
                                dict(buckets=[0, 1 << 17]), dict(sms=0), dict(buckets=[0] * 65537)])
def test_bad_plans(cplib, kw):
    a = dict(cu=[0, 5], heads=2, prefix=0, buckets=None, sms=152)
    a.update(kw)
    with pytest.raises(CpError):
        build_plan(a["cu"], a["heads"], a["prefix"], True, a["buckets"], a["sms"])


A, ODD = 4096, 4097


def _call(direction="fwd", plan=None, plan_d=A, dt=1, T=5, H=2, Hkv=1, d=64, scale=0.125, ws=A, ws_bytes=1 << 20,
          out_lo=None, dbias=None, score=None, null_score=False, swap=None, grad_dt=0, dbias_dt=0, **over):
    """Status of a call on stand-in pointers; a refused call never touches them."""
    plan = build_plan([0, 5], 2, 0, False, [0, 1, 1, 2], 152)[0] if plan is None else plan
    s = B.ScoreDesc()
    s.softcap, s.n_buckets, s.bias_stride_h, s.bias_stride_b = 0.0, 3, 3, 1
    for k, v in {**(score or {}), **over}.items():
        setattr(s, k, v)
    p = [A] * (5 if direction == "fwd" else 9)      # q k v out lse | q k v out lse dout dq dk dv
    if swap is not None:
        p[swap[0]] = swap[1]
    vp = [ctypes.c_void_p(x) if x is not None else None for x in p]
    sref = None if null_score else ctypes.byref(s)
    shape = (dt, T, H, Hkv, d, sref, scale)
    host = _host(plan) if not isinstance(plan, int) else ctypes.c_void_p(plan)
    if direction == "fwd":
        return B.lib().cp_attn_scored_fwd(host, plan_d, *vp[:3], *shape, *vp[3:], out_lo, ws, ws_bytes, None)
    return B.lib().cp_attn_scored_bwd(host, plan_d, *vp[:4], out_lo, *vp[4:6], *shape, *vp[6:], grad_dt, dbias, dbias_dt,
                                      ws, ws_bytes, None)


BAD = [(dict(plan=bytearray(256)), 1), (dict(null_score=True), 1), (dict(dt=5), 3), (dict(T=6), 2), (dict(H=4), 2),
       (dict(Hkv=0), 2), (dict(H=2, Hkv=3), 2), (dict(d=96), 2), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
       (dict(scale=float("nan")), 1), (dict(softcap=-1.0), 1), (dict(softcap=float("inf")), 1),
       (dict(softcap=1e-5), 1), (dict(softcap=1e6), 1), (dict(slopes=A, rel_bias=A), 1), (dict(slopes=ODD), 4),
       (dict(rel_bias=A, bias_dtype=4), 3), (dict(rel_bias=A, n_buckets=2), 2), (dict(rel_bias=ODD, bias_dtype=1), 4),
       (dict(plan_d=None), 1), (dict(plan_d=A + 16), 4), (dict(ws=None), 5), (dict(ws_bytes=100), 5),
       (dict(ws=A + 16), 4), (dict(dt=0, out_lo=A), 3), (dict(out_lo=A + 8), 4)]


@pytest.mark.parametrize("direction", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,status", BAD)
def test_bad_calls(cplib, direction, kw, status):
    assert _call(direction, **kw) == status
    assert B.lib().cp_last_error()


def test_bad_pointers(cplib):
    for direction, n in (("fwd", 5), ("bwd", 9)):
        for i in range(n):
            assert _call(direction, swap=(i, None)) == 1
            assert _call(direction, swap=(i, A + 8)) == 4
    assert _call("bwd", dbias=A) == 1                       # no rel_bias to differentiate
    assert _call("bwd", rel_bias=A, dbias=ODD) == 4
    assert _call("bwd", grad_dt=7) == 3
    assert _call("bwd", dt=0, grad_dt=1) == 3               # bf16 gradients of fp32 inputs
    assert _call("bwd", rel_bias=A, dbias=A, dbias_dt=5) == 3
    need = B.lib().cp_attn_scored_bwd_workspace_size(_host(build_plan([0, 5], 2, 0, False, [0, 1, 1, 2], 152)[0]),
                                                     1, 1, 64, 0.125, 1)
    assert _call("bwd", grad_dt=1, ws_bytes=need - 1) == 5
    plain = build_plan([0, 5], 2, 0, False, None, 152)[0]
    assert _call("fwd", plan=plain, rel_bias=A) == 1        # a plan without buckets
    assert _call("fwd", plan=0) == 1


def test_no_tokens(cplib):
    empty = build_plan([0, 0], 2, 0, False, None, 152)[0]
    assert _call("fwd", plan=empty, T=0, plan_d=None, ws=None, swap=(0, None)) == 0
    assert _call("bwd", plan=empty, T=0, plan_d=None, ws=None, swap=(0, None)) == 0


def test_python_refuses_cpu_tensors():
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_fwd
    with pytest.raises(CpError):
        ScorePlan([0, 4], 2, device="cpu")
    q = torch.zeros(4, 2, 64)
    with pytest.raises(CpError):
        cp_attn_scored_fwd(q, q, q, None, 0.125)


def test_more_heads_than_a_grid_holds(cplib):
    assert build_plan([0, 5], 65535, 0, False, None, 152)[1] == 5
    with pytest.raises(CpError):
        build_plan([0, 5], 65536, 0, False, None, 152)


def _cut(plan, dtype, d=64):
    """Bytes that a forward needs for partial results, per element of a row."""
    block = (ctypes.c_char * len(plan)).from_buffer(plan)
    return B.lib().cp_attn_scored_fwd_workspace_size(block, dtype, 1, d, 0.125)


@pytest.mark.parametrize("lens,prefix,H", [([3000], 0, 1), ([1025, 0, 2000], 300, 2), ([4999, 1], 1, 4),
                                           ([2048, 130], [2048, 5], 1), ([129] * 20 + [5000], 7, 3)])
@pytest.mark.parametrize("both", [False, True])
def test_cut_plans_cover_the_visible_pairs(cplib, lens, prefix, H, both):
    """Few heads: long runs are cut into parts, which still meet every pair once."""
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    pre = [min(prefix, n) for n in lens] if isinstance(prefix, int) else prefix
    want = sum(n * (n + 1) // 2 + (p * (p - 1) // 2 if both else 0) for n, p in zip(lens, pre))
    for sms in (1, 16, 152, 4096):
        plan, T = build_plan(cu, H, pre, both, None, sms)
        assert _pairs(plan) == [want] * 3
        if sms != 16:   # one multiprocessor has nobody to share with
            assert (_cut(plan, 1) > 256) == (sms > 16)
    with pytest.raises(CpError):
        build_plan(cu, H, pre, both, None, 4097)


def test_plans_that_fill_the_gpu_are_not_cut(cplib):
    for lens, H in (([4096], 16), ([8192], 8), ([2048, 1531, 700], 12), ([512], 8), ([40] * 300, 4)):
        plan, _ = build_plan(np.concatenate([[0], np.cumsum(lens)]).tolist(), H, 0, False, None, 152)
        assert _cut(plan, 1) == 256   # the status alone


def test_buckets_of_any_whole_numbers(cplib):
    want, _ = build_plan([0, 9], 1, 0, False, [0, 1, 1, 2], 152)
    for same in (np.array([0, 1, 1, 2]), torch.tensor([0, 1, 1, 2]), (0, True, 1, 2)):
        assert build_plan([0, 9], 1, 0, False, list(same), 152)[0] == want
    for bad in ([0, 0.5], [0, 1 << 40], ["0"]):
        with pytest.raises(CpError):
            build_plan([0, 9], 1, 0, False, bad, 152)


@pytest.mark.parametrize("n,far", [(2, 2), (3, 9), (8, 16), (32, 128), (33, 100), (64, 4096)])
def test_relative_buckets_equal_their_formula(n, far):
    import math
    exact = n // 2
    want = [d if d < exact else
            min(n - 1, exact + int(math.log(d / exact) / math.log(far / exact) * (n - exact) + 1e-9))
            for d in range(far + 1)]
    assert relative_buckets(n, far) == want
